"""Products of 8-bit integers whose waits run out: the kernel returns, says so in the device
status word, and leaves a device that computes.

gptq_selftest_int8_timeout makes some threads of a product take a wait for run out while the
others go on, which is what two threads do that look at the same barrier just before and
just behind the end of their second.  A kernel in which those that go on wait for those that
left never returns.
"""

import pytest

from test_gpu_int8 import F32, assert_close, codes8, layer8, product

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

WARP, SUMS, THREAD = 1, 2, 3
TIMEOUT = 5

# (n, r, d), several tiles to a CTA: single CTAs, pairs, pairs with the tokens' last tile ragged
MANY_TILES = [(8, 80000, 32), (40, 60000, 96), (256, 60000, 32), (300, 40000, 256)]
IDS = ["n{}_r{}_d{}".format(*s) for s in MANY_TILES]


def give_up(lib, shape, what):
    """The status after a product that gives up, and the same product afterwards."""
    import post_weight_quantization_19_b200 as g
    n, r, d = shape
    (x, xs), (w, ws) = codes8(n, d, n), layer8(r, d, r)
    y = torch.zeros((n, r), device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert g.gptq_check_device_status() == 0
    assert lib.gptq_selftest_int8_timeout(x.data_ptr(), xs.data_ptr(), n, w.data_ptr(), ws.data_ptr(), r, d, what,
                                          y.data_ptr(), stream) == 0
    status = g.gptq_check_device_status()
    assert g.gptq_check_device_status() == 0
    whole = g.gptq_int8_linear(x, xs, w, ws, dtype=F32)
    assert_close(whole, *product(x, xs, w, ws))
    assert g.gptq_check_device_status() == 0
    return status, y, whole


@pytest.mark.parametrize("shape", MANY_TILES, ids=IDS)
def test_a_warp_that_gives_up_leaves_no_other_waiting(lib, shape):
    status, y, whole = give_up(lib, shape, WARP)
    assert status == TIMEOUT
    # what was written is right, and something was not
    written = y != 0
    assert bool(written.any()) and torch.equal(y[written], whole[written])
    assert int(written.sum()) < int((whole != 0).sum())


@pytest.mark.parametrize("shape", MANY_TILES, ids=IDS)
def test_a_thread_that_gives_up_alone_is_reported(lib, shape):
    # its warp writes nothing then, and the caller has to hear of it
    status, y, whole = give_up(lib, shape, THREAD)
    assert int((y != 0).sum()) < int((whole != 0).sum())
    assert status == TIMEOUT


# columns split over 4 and 8 CTAs, their sums beside the ring of stages (up to 32 tokens) and in it
@pytest.mark.parametrize("shape", [(1, 300, 4096), (20, 3000, 4096), (10, 4608, 16384), (64, 300, 8192), (256, 130, 16384)],
                         ids="n{0[0]}_r{0[1]}_d{0[2]}".format)
def test_a_cta_that_gives_up_on_sums_stays_until_they_landed(lib, shape):
    # (the others push their sums to its memory, which must not have gone)
    for _ in range(5):
        status, y, whole = give_up(lib, shape, SUMS)
        assert status == TIMEOUT
        written = y != 0
        assert bool(written.any()) and torch.equal(y[written], whole[written])
        assert int(written.sum()) < int((whole != 0).sum())


def test_a_product_without_such_a_wait_is_computed(lib):
    for what in (WARP, SUMS, THREAD):
        status, y, whole = give_up(lib, (3, 64, 96), what)
        assert status == 0 and torch.equal(y, whole)
