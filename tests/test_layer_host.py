"""Host side of the operators that run a calibrated layer: sizes, refusals before any launch, empty calls, and the
reference's own tile order (no GPU)."""
import numpy as np
import pytest

from tests import layer_ref as ref

FAKE = 0x10000000  # never dereferenced: validation fails first, or there is nothing to do


def _lh():
    import scale_calibration_b200 as lh
    return lh


def refuse(fn, ok, cases):
    lh = _lh()
    for over, want in cases:
        assert fn(**dict(ok, **over)) == want, over
        assert lh.lh_last_error_message() != "", over


def test_route_refusals():
    lh = _lh()
    ok = dict(ids=FAKE, n_tok=10, k=4, n_experts=64, offsets=FAKE + 4096, order=FAKE + 8192, pos=FAKE + 16384, stream=0,
              check=False)
    refuse(lh.lh_route_tokens, ok, [
        (dict(ids=0), 1), (dict(offsets=0), 1), (dict(order=0), 1), (dict(pos=0), 1), (dict(n_tok=-1), 1),
        (dict(k=0), 1), (dict(n_experts=0), 1), (dict(n_experts=1025), 2), (dict(n_tok=1 << 30, k=2), 2),
        (dict(k=1 << 31), 2), (dict(pos=FAKE + 8192), 1), (dict(pos=FAKE), 1), (dict(order=FAKE), 1),
    ])


def test_gather_refusals():
    lh = _lh()
    ok = dict(X=FAKE, dtype=lh.LH_BF16, n_tok=10, c=100, ld_x=104, order=FAKE, k=2, n_rows=20, Xs=FAKE + 65536,
              ld_xs=104, stream=0, check=False)
    refuse(lh.lh_gather_tokens, ok, [
        (dict(X=0), 1), (dict(order=0), 1), (dict(Xs=0), 1), (dict(Xs=FAKE), 1), (dict(n_tok=-1), 1), (dict(c=-1), 1),
        (dict(k=0), 1), (dict(n_rows=-1), 1), (dict(ld_x=96), 1), (dict(ld_xs=96), 1), (dict(ld_x=100), 3),
        (dict(ld_xs=100), 3), (dict(X=FAKE + 8), 3), (dict(Xs=FAKE + 65544), 3), (dict(dtype=5), 2),
    ])
    for over in (dict(n_tok=0), dict(c=0), dict(n_rows=0)):
        assert lh.lh_gather_tokens(**dict(ok, **over)) == 0


def test_combine_refusals():
    lh = _lh()
    ok = dict(Ys=FAKE, dtype=lh.LH_F32, n_rows=20, c=30, ld_ys=32, pos=FAKE, weights=None, n_tok=10, k=2,
              Y=FAKE + 65536, ld_y=32, stream=0, check=False)
    refuse(lh.lh_combine_tokens, ok, [
        (dict(Ys=0), 1), (dict(pos=0), 1), (dict(Y=0), 1), (dict(Y=FAKE), 1), (dict(n_rows=-1), 1), (dict(c=-1), 1),
        (dict(n_tok=-1), 1), (dict(k=0), 1), (dict(n_tok=1 << 30, k=2), 2), (dict(ld_ys=29), 1), (dict(ld_y=29), 1),
        (dict(ld_ys=33), 3), (dict(ld_y=30), 3), (dict(Ys=FAKE + 4), 3), (dict(dtype=-1), 2),
    ])
    for over in (dict(n_tok=0), dict(c=0)):
        assert lh.lh_combine_tokens(**dict(ok, **over)) == 0


def test_combine_gradient_refusals():
    lh = _lh()
    ok = dict(dY=FAKE, dtype=lh.LH_F32, n_tok=10, k=2, c=30, ld_dy=32, Ys=FAKE + 65536, ld_ys=32, n_rows=20, pos=FAKE,
              weights=None, dYs=FAKE + 131072, ld_dys=32, dweights=FAKE, stream=0, check=False)
    refuse(lh.lh_combine_tokens_grad, ok, [
        (dict(dY=0), 1), (dict(pos=0), 1), (dict(Ys=0), 1), (dict(dYs=0, dweights=0), 1), (dict(dYs=FAKE), 1),
        (dict(dYs=FAKE + 65536), 1), (dict(n_rows=-1), 1), (dict(c=-1), 1), (dict(k=0), 1), (dict(n_tok=-2), 1),
        (dict(ld_dy=28), 1), (dict(ld_ys=28), 1), (dict(ld_dys=28), 1), (dict(ld_dy=30), 3), (dict(ld_ys=31), 3),
        (dict(ld_dys=33), 3), (dict(dtype=9), 2), (dict(n_tok=1 << 30, k=2), 2),
    ])
    assert lh.lh_combine_tokens_grad(**dict(ok, n_tok=0)) == 0
    assert lh.lh_combine_tokens_grad(**dict(ok, c=0, dweights=0)) == 0


def test_scale_tile_sizes_and_refusals():
    lh = _lh()
    assert lh.lh_nvfp4_weight_scale_bytes(1, 128, 64) == 512
    assert lh.lh_nvfp4_weight_scale_bytes(3, 129, 80) == 3 * 2 * 2 * 512
    assert lh.lh_nvfp4_weight_scale_bytes(0, 128, 64) == 0 and lh.lh_nvfp4_weight_scale_bytes(1, 128, 40) == 0
    assert lh.lh_nvfp4_token_scale_bytes(1, 64, 1) == 512
    assert lh.lh_nvfp4_token_scale_bytes(300, 128, 5) == (2 + 5) * 2 * 512
    assert lh.lh_nvfp4_token_scale_bytes(-1, 64, 1) == 0 and lh.lh_nvfp4_token_scale_bytes(1, 64, 0) == 0
    ok = dict(block_scales=FAKE, n_mats=1, c_out=128, c_in=64, tiles=FAKE + 65536, stream=0, check=False)
    refuse(lh.lh_nvfp4_tile_scales, ok, [
        (dict(block_scales=0), 1), (dict(tiles=0), 1), (dict(n_mats=0), 1), (dict(c_out=-1), 1), (dict(c_in=24), 2),
        (dict(tiles=FAKE + 65544), 3), (dict(tiles=FAKE), 1),
    ])
    assert lh.lh_nvfp4_tile_scales(**dict(ok, c_out=0)) == 0


@pytest.mark.parametrize("seed", range(20))
def test_groups_do_not_share_tiles_and_fit_the_size(seed):
    # the places that the header gives groups: first tile offsets[g] / 128 + g, ceil(rows / 128) tiles each
    lh = _lh()
    rng = np.random.default_rng(seed)
    G = int(rng.integers(1, 40))
    counts = rng.choice([0, 1, 2, 31, 127, 128, 129, 255, 256, 257, 1000], G)
    off = np.concatenate([[0], np.cumsum(counts)]) + int(rng.integers(0, 300))
    n = int(off[-1]) + int(rng.integers(0, 300))
    used = np.zeros(lh.lh_nvfp4_token_scale_bytes(n, 64, G) // 512, int)
    for g in range(G):
        t0 = off[g] // 128 + g
        assert t0 + -(-counts[g] // 128) <= len(used)
        used[t0:t0 + -(-counts[g] // 128)] += 1
    assert used.max(initial=0) <= 1


def test_the_references_tiles_undo():
    rng = np.random.default_rng(0)
    for n, J, first, group in [(1, 1, 0, 0), (130, 9, 300, 4), (257, 4, 0, 2)]:
        codes = rng.integers(1, 127, (n, J)).astype(np.uint8)
        t = ref.tile(codes, first, group)
        back = ref.untile(t, n, J, first, group)
        assert np.array_equal(back[:, :J], codes) and (back[:, J:] == 0).all()


def test_the_references_route():
    ids = np.array([[2, 0], [-1, 2], [5, 0]], np.int32)
    off, order, pos = ref.route(ids, 3)
    assert off.tolist() == [0, 2, 2, 4] and order.tolist() == [1, 5, 0, 3, -1, -1]
    assert pos.tolist() == [2, 0, -1, 3, -1, 1]


def test_quantize_tokens_refusals():
    lh = _lh()
    ok = dict(X=FAKE, x_dtype=lh.LH_BF16, n_src=10, c_in=64, ld_x=64, rows=None, row_div=1, n_rows=10, offsets=None,
              n_groups=1, global_amax=None, packed=FAKE + 65536, scale_tiles=FAKE + 131072, token_scale=FAKE + 262144,
              X_out=None, out_dtype=lh.LH_BF16, stream=0, check=False)
    refuse(lh.lh_quantize_tokens, ok, [
        (dict(X=0), 1), (dict(packed=0), 1), (dict(scale_tiles=0), 1), (dict(token_scale=0), 1), (dict(n_src=-1), 1),
        (dict(n_rows=-1), 1), (dict(n_groups=0), 1), (dict(n_groups=2), 1), (dict(row_div=0), 1), (dict(row_div=2), 1),
        (dict(n_rows=11), 1), (dict(c_in=40, ld_x=40), 2), (dict(ld_x=48), 1), (dict(ld_x=68), 3), (dict(X=FAKE + 8), 3),
        (dict(packed=FAKE + 65544), 3), (dict(scale_tiles=FAKE + 131080), 3), (dict(X_out=FAKE + 8), 3),
        (dict(X_out=FAKE), 1), (dict(packed=FAKE), 1), (dict(scale_tiles=FAKE + 65536), 1), (dict(x_dtype=3), 2),
        (dict(X_out=FAKE + 524288, out_dtype=3), 2), (dict(c_in=(1 << 28) + 16, ld_x=(1 << 28) + 16), 2),
        (dict(n_src=1 << 31, n_rows=1 << 31), 2), (dict(row_div=1 << 31, rows=FAKE), 2),
    ])
    for over in (dict(n_rows=0), dict(c_in=0)):
        assert lh.lh_quantize_tokens(**dict(ok, **over)) == 0


def test_matmul_refusals():
    lh = _lh()
    ok = dict(X_packed=FAKE, X_scales=FAKE, X_gscale=FAKE, W_packed=FAKE, W_scales=FAKE, W_gscale=FAKE, offsets=None,
              n_groups=1, n_rows=10, c_out=100, c_in=64, Y=FAKE + 65536, out_dtype=lh.LH_F32, ld_y=100, stream=0,
              check=False)
    refuse(lh.lh_nvfp4_matmul, ok, [
        (dict(X_packed=0), 1), (dict(X_scales=0), 1), (dict(X_gscale=0), 1), (dict(W_packed=0), 1),
        (dict(W_scales=0), 1), (dict(W_gscale=0), 1), (dict(Y=0), 1), (dict(n_rows=-1), 1), (dict(c_out=-1), 1),
        (dict(n_groups=0), 1), (dict(n_groups=2), 1), (dict(c_in=48), 2), (dict(c_in=0), 2), (dict(ld_y=96), 1),
        (dict(ld_y=101), 3), (dict(Y=FAKE + 65540), 3), (dict(X_packed=FAKE + 8), 3), (dict(W_scales=FAKE + 8), 3),
        (dict(Y=FAKE), 1), (dict(out_dtype=2), 2), (dict(n_rows=(1 << 31) - 1), 2),
        (dict(offsets=FAKE, n_groups=1 << 20, c_out=4096, ld_y=4096), 2),
    ])
    for over in (dict(n_rows=0), dict(c_out=0)):
        assert lh.lh_nvfp4_matmul(**dict(ok, **over)) == 0


def test_linear_refusals():
    lh = _lh()
    need = lh.lh_nvfp4_linear_workspace_bytes(10, 64, 1)
    assert need == 10 * 32 + 192 + 512 + 256
    assert lh.lh_nvfp4_linear_workspace_bytes(0, 64, 1) == 0 and lh.lh_nvfp4_linear_workspace_bytes(1, 48, 1) == 0
    ok = dict(X=FAKE, x_dtype=lh.LH_F32, n_src=10, c_in=64, ld_x=64, rows=None, row_div=1, n_rows=10, offsets=None,
              n_groups=1, global_amax=None, W_packed=FAKE, W_scales=FAKE, W_gscale=FAKE, c_out=100, Y=FAKE + 65536,
              out_dtype=lh.LH_F32, ld_y=100, workspace=FAKE + 131072, workspace_bytes=need, stream=0, check=False)
    refuse(lh.lh_nvfp4_linear, ok, [
        (dict(workspace=0), 4), (dict(workspace_bytes=need - 1), 4), (dict(workspace=FAKE + 131088), 3),
        (dict(X=0), 1), (dict(W_packed=0), 1), (dict(Y=0), 1), (dict(Y=FAKE), 1), (dict(x_dtype=7), 2),
        (dict(out_dtype=7), 2), (dict(c_in=48, ld_x=48), 2), (dict(ld_x=60), 1), (dict(ld_x=66), 3),
        (dict(X=FAKE + 4), 3), (dict(row_div=3), 1), (dict(n_rows=11, workspace_bytes=1 << 20), 1), (dict(n_groups=3), 1),
        (dict(ld_y=99), 1), (dict(ld_y=102), 3), (dict(W_scales=FAKE + 4), 3), (dict(n_src=-1), 1),
    ])
    for over in (dict(n_rows=0), dict(c_out=0)):
        assert lh.lh_nvfp4_linear(**dict(ok, **over)) == 0
