"""How the products of 8-bit integers are launched, over their range of sizes and without a GPU
(gptq_int8_plan): what the kernels take for granted of their launches."""

import ctypes
import random

SMEM_CTA = 227 * 1024      # most shared memory of a CTA
SMEM_SM = 228 * 1024       # of an SM, 1 KB of it reserved for each CTA
COLUMNS_SM = 512           # of tensor memory


def plan(lib, n, r, d, gated, sms=148):
    out = (ctypes.c_int64 * 8)()
    assert lib.gptq_int8_plan(n, r, d, gated, sms, out) == 0, (n, r, d, gated, sms)
    return dict(zip(("pairs", "ctas", "cluster", "tokens", "rows", "stages", "columns", "smem"), out))


def sizes(count=20000):
    """Sizes over the whole range, and next to where the kernels change."""
    rng = random.Random(5)
    for _ in range(count):
        n = rng.choice([1, 2, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 127, 128, 129, 144, 145, 255, 256, 257,
                        int(2 ** rng.uniform(0, 14)), rng.randint(1, 300)])
        r = rng.choice([rng.randint(1, 300), int(2 ** rng.uniform(0, 19)), 128 * rng.randint(1, 160)])
        d = 32 * rng.choice([rng.randint(1, 40), int(2 ** rng.uniform(0, 11)), 4 * rng.randint(1, 512)])
        yield n, r, min(d, 65536), rng.randint(0, 1), rng.choice([148, 148, 148, 132, 64, 2])


def test_refusals(lib):
    out = (ctypes.c_int64 * 8)()
    for bad in ((0, 8, 64, 0, 148), (8, 0, 64, 0, 148), (-1, 8, 64, 0, 148), (8, -1, 64, 0, 148), (8, 8, 40, 0, 148),
                (8, 8, 0, 0, 148), (8, 8, 65568, 0, 148), (1 << 31, 8, 64, 0, 148), (8, 8, 64, 0, 1), (8, 8, 64, 0, 4097)):
        assert lib.gptq_int8_plan(*bad, out) == 1, bad
    assert lib.gptq_int8_plan(8, 8, 64, 0, 148, None) == 1


def test_single_ctas_take_all_tokens_in_one_tile(lib):
    # that kernel knows one tile of tokens, two accumulators where k is not split
    seen = set()
    for n, r, d, gated, sms in sizes():
        p = plan(lib, n, r, d, gated, sms)
        layers, case = 1 + gated, (n, r, d, gated, sms, p)
        assert 1 <= p["stages"] <= 12 and p["smem"] <= SMEM_CTA, case
        if p["pairs"]:
            assert n > 64 and p["tokens"] == 256 and p["cluster"] == 2, case
            assert 2 <= p["ctas"] <= sms and p["ctas"] % 2 == 0 and p["stages"] >= 4, case
            assert p["rows"] * layers <= 256 and p["rows"] * layers % 32 == 0 and p["columns"] == 512, case
            continue
        seen.add((gated, p["cluster"], n > 64))
        tiles = -(-r // p["rows"])
        assert n <= p["tokens"] < n + 16 and p["tokens"] % 16 == 0 and p["tokens"] <= 256 // layers, case
        assert 8 <= p["rows"] <= 128 and p["rows"] % 8 == 0, case
        accumulators = 1 if p["cluster"] > 1 else 2
        assert p["columns"] in (32, 64, 128, 256) and p["columns"] >= accumulators * layers * p["tokens"], case
        if p["cluster"] > 1:
            assert p["rows"] == 128 and p["ctas"] == tiles * p["cluster"], case
            assert -(-d // 128) >= 2 * p["cluster"], case    # every CTA has columns
        else:
            assert n <= 64 and p["ctas"] <= min(tiles, 2 * sms), case
    assert {(0, 8, False), (0, 4, False), (1, 8, False), (1, 4, False), (1, 2, False), (0, 1, False), (1, 1, False),
            (0, 8, True), (1, 8, True)} <= seen, sorted(seen)


def test_ctas_that_fit_on_an_sm_together_find_their_tensor_memory(lib):
    # Each CTA takes its columns without a limit on the wait, and CTAs of a cluster then wait for
    # each other: if those that shared memory lets onto an SM together, of whatever streams'
    # kernels, could ask for more columns than it has, two clusters could hold what the
    # other waits for.
    least = {}   # columns -> least shared memory that goes with them, and where
    for n, r, d, gated, sms in sizes():
        p = plan(lib, n, r, d, gated, sms)
        held = p["smem"] + 1024
        if held < least.get(p["columns"], (1 << 30,))[0]:
            least[p["columns"]] = held, (n, r, d, gated, sms)
    assert set(least) == {32, 64, 128, 256, 512}

    def most(room, columns):   # columns that the CTAs in this much shared memory can ask for
        return max([0] + [c + most(room - held, c) for c, (held, _) in least.items() if held <= room and c <= columns])

    assert most(SMEM_SM, COLUMNS_SM) <= COLUMNS_SM, least
