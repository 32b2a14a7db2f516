"""What the operators that run a calibrated layer accept and refuse at the ends of their ranges (no GPU)."""
import pytest

FAKE = 0x10000000  # never dereferenced: validation fails first, or there is nothing to do
MOST = (1 << 31) - 513  # flat slots, rows


def _lh():
    import scale_calibration_b200 as lh
    return lh


@pytest.mark.parametrize("n,k", [(MOST + 1, 1), (1, MOST + 1), ((1 << 31) - 1, 1), (1, (1 << 31) - 1), (1 << 28, 8),
                                 (715827712, 3)])
def test_flat_indices_that_a_32_bit_counter_would_step_past_are_refused(n, k):
    lh = _lh()
    assert lh.lh_route_tokens(FAKE, n, k, 4, FAKE + 4096, FAKE + 8192, FAKE + 16384, 0, False) == 2
    assert lh.lh_combine_tokens(FAKE, lh.LH_F32, 8, 8, 8, FAKE, None, n, k, FAKE + 65536, 8, 0, False) == 2
    assert lh.lh_combine_tokens_grad(FAKE, lh.LH_F32, n, k, 8, 8, FAKE + 65536, 8, 8, FAKE, None, FAKE + 131072, 8, FAKE,
                                     0, False) == 2
    # one slot less is no matter of sizes: other checks answer
    if n == MOST + 1:
        assert lh.lh_route_tokens(0, n - 1, k, 4, FAKE + 4096, FAKE + 8192, FAKE + 16384, 0, False) == 1


@pytest.mark.parametrize("c_in", [(1 << 28) + 32, (1 << 31) - 1024])
def test_products_longer_than_any_quantised_token_are_refused(c_in):
    # a tile of 2^31 columns takes more than two seconds, longer than the kernel's waits for it
    lh = _lh()

    def call(c, n=0):
        return lh.lh_nvfp4_matmul(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 1, n, 8, c, FAKE + 65536, lh.LH_F32, 8, 0, False)

    assert call(c_in) == 2 and call(1 << 28) == 0


def linear_args(**over):
    lh = _lh()
    a = dict(X=FAKE, x_dtype=lh.LH_F32, n_src=10, c_in=64, ld_x=64, rows=None, row_div=1, n_rows=0, offsets=None,
             n_groups=1, global_amax=None, W_packed=FAKE + 262144, W_scales=FAKE + 524288, W_gscale=FAKE + 589824,
             c_out=100, Y=FAKE + 65536, out_dtype=lh.LH_F32, ld_y=100, workspace=FAKE + 131072, workspace_bytes=4096,
             stream=0, check=False)
    a.update(over)
    return a


@pytest.mark.parametrize("n_rows", [0, 1, 10])
def test_linear_refuses_an_output_over_its_weights_or_workspace(n_rows):
    # whichever kernel the sizes choose: one row is quantised by the product, ten are not
    lh = _lh()
    assert lh.lh_nvfp4_linear(**linear_args()) == 0
    for y in ("X", "W_packed", "W_scales", "workspace"):
        a = linear_args(n_rows=n_rows)
        a["Y"] = a[y]
        assert lh.lh_nvfp4_linear(**a) == 1, y
        assert "alias" in lh.lh_last_error_message()


def test_empty_calls_take_null_arrays():
    # an empty tensor's pointer is NULL
    lh = _lh()
    t = lh.LH_BF16
    assert lh.lh_gather_tokens(0, t, 0, 64, 64, 0, 2, 0, 0, 64, 0, False) == 0
    assert lh.lh_gather_tokens(0, t, 0, 64, 64, FAKE, 2, 5, FAKE, 64, 0, False) == 0
    assert lh.lh_gather_tokens(FAKE, t, 9, 64, 64, 0, 2, 0, 0, 64, 0, False) == 0
    assert lh.lh_combine_tokens(0, t, 0, 64, 64, 0, None, 0, 2, 0, 64, 0, False) == 0
    assert lh.lh_combine_tokens_grad(0, t, 0, 2, 64, 64, 0, 64, 0, 0, None, 0, 64, 0, 0, False) == 0
    assert lh.lh_combine_tokens_grad(FAKE, t, 3, 2, 64, 64, 0, 64, 0, FAKE, None, 0, 64, 0, 0, False) == 0
    for n_src, n_rows in ((0, 0), (9, 0)):
        x = FAKE if n_src else 0
        assert lh.lh_quantize_tokens(x, t, n_src, 64, 64, None, 1, n_rows, None, 1, None, 0, 0, 0, None, t, 0, False) == 0
        assert lh.lh_nvfp4_linear(x, t, n_src, 64, 64, None, 1, n_rows, None, 1, None, FAKE, FAKE, FAKE, 8, 0, t, 8, 0, 0,
                                  0, False) == 0
    assert lh.lh_nvfp4_matmul(0, 0, 0, FAKE, FAKE, FAKE, None, 1, 0, 8, 64, 0, t, 8, 0, False) == 0
    assert lh.lh_nvfp4_matmul(FAKE, FAKE, FAKE, 0, 0, FAKE, None, 1, 4, 0, 64, 0, t, 8, 0, False) == 0
    assert lh.lh_nvfp4_tile_scales(0, 2, 0, 64, 0, 0, False) == 0
    assert lh.lh_accumulate_hessian(0, t, 0, 64, 64, None, 1, FAKE, 0, 0, 0, False) == 0
    assert lh.lh_accumulate_hessian_noalloc(0, t, 0, 64, 64, None, 1, FAKE, 0, False) == 0


def test_null_arrays_that_have_elements_are_refused():
    lh = _lh()
    t = lh.LH_BF16
    assert lh.lh_gather_tokens(0, t, 1, 64, 64, FAKE, 2, 5, FAKE, 64, 0, False) == 1
    assert lh.lh_combine_tokens(FAKE, t, 4, 64, 64, FAKE, None, 1, 2, 0, 64, 0, False) == 1
    assert lh.lh_combine_tokens(0, t, 4, 64, 64, FAKE, None, 1, 2, FAKE, 64, 0, False) == 1
    assert lh.lh_combine_tokens_grad(FAKE, t, 1, 2, 64, 64, 0, 64, 4, FAKE, None, 0, 64, FAKE, 0, False) == 1
    assert lh.lh_quantize_tokens(0, t, 1, 64, 64, None, 1, 1, None, 1, None, FAKE, FAKE + 4096, FAKE, None, t, 0, False) == 1
    assert lh.lh_nvfp4_matmul(FAKE, FAKE, 0, FAKE, FAKE, FAKE, None, 1, 1, 8, 64, FAKE + 4096, t, 8, 0, False) == 1
    assert lh.lh_nvfp4_tile_scales(0, 2, 1, 64, FAKE, 0, False) == 1
    assert lh.lh_accumulate_hessian(0, t, 1, 64, 64, None, 1, FAKE, FAKE, 1 << 20, 0, False) == 1


def test_wait_probe_refusals():
    lh = _lh()
    for us in (0, -1, 1000001):
        assert lh.lh_debug_nvfp4_wait_timeout(us, 0, 0, False) == 1
