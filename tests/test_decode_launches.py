"""The few-token layer's launches, recorded by a host program that stands in for the HIP runtime: the LDS limit
that a kernel is given holds for every call's size, so that two threads' calls cannot lower each other's."""
import pytest

from launch_recorder import record

MAIN = r"""
int main()
{
    static uint8_t none[256];
    std::printf("[");
    const int sizes[][5] = {SIZES};                       // d, f, E, k, T
    for (auto& s : sizes)
        for (int dtype = 0; dtype < 3; ++dtype) {
            moe::DecodeLaunch D{};
            D.d = s[0], D.f = s[1], D.E = s[2], D.k = s[3], D.T = s[4], D.dtype = dtype;
            D.L = moe::decode_ws(D.d, D.f, D.E, D.k, D.T);
            D.expert_stride = (uint64_t)27 * D.d * D.f / 16;
            D.ws = none, D.blob = none;
            if (launch_decode_route(D, 0) != hipSuccess || launch_decode_products(D, 0) != hipSuccess ||
                launch_decode_combine(D, 0) != hipSuccess) return 1;
        }
    std::printf("]\n");
    return 0;
}
"""

# (size, launches of a call): the fused down and combine saves one
RULE = [((512, 256, 8, 2, 1), 2), ((128, 2048, 8, 2, 2), 2), ((2048, 4096, 16, 1, 4), 2), ((2048, 4096, 16, 1, 5), 3),
        ((2048, 768, 64, 7, 1), 2), ((2048, 768, 64, 8, 1), 3), ((64, 64, 64, 8, 1), 2), ((64, 64, 64, 9, 1), 3),
        ((64, 16384, 16, 4, 1), 3)]                       # its h is past the LDS of the rule
# (size, threads of a gate/up workgroup)
WAVES = [((2048, 768, 128, 8, 2), 512), ((2048, 768, 128, 8, 3), 256), ((2048, 512, 128, 8, 4), 512), ((2080, 768, 128, 8, 5), 512),
         ((4096, 1536, 256, 8, 4), 512), ((1184, 352, 60, 4, 16), 256)]
SIZES = [s for s, _ in RULE + WAVES] + [(d, f, E, k, T) for d, f in [(64, 96), (2048, 768), (4096, 1536), (1184, 352), (16384, 1024), (1024, 16384), (16384, 16384)]
         for E, k in [(1, 1), (8, 2), (128, 8)] for T in (1, 2, 24, 128)]


@pytest.fixture(scope="module")
def events(tmp_path_factory):
    main = MAIN.replace("SIZES", ", ".join("{%d, %d, %d, %d, %d}" % s for s in SIZES))
    return record(tmp_path_factory.mktemp("launches"), "moe_decode.h", "moe_decode.hip", main)


def test_a_kernels_lds_limit_is_the_same_for_every_size(events):
    limits = {}
    for kind, f, v, *_ in events:
        if kind == "limit":
            limits.setdefault(f, set()).add(v)
    assert limits
    assert all(len(v) == 1 for v in limits.values()), limits


def test_every_launch_is_within_its_kernels_limit(events):
    limit, seen = {}, 0
    for kind, f, v, *grid in events:
        if kind == "limit":
            limit[f] = v
            assert v <= 160 << 10
        else:
            assert v <= limit.get(f, 16 << 10), (f, v)
            assert grid[0] >= 1 and 1 <= grid[1] <= 65535 and grid[2] <= 1024
            seen += 1
    assert seen > len(SIZES) * 3


def test_which_calls_fuse_the_down_product_and_the_combine(events):
    """One launch for a few pairs' down product and combine; gate/up before it, and nothing else."""
    it = iter([e for e in events if e[0] == "launch"])
    for size, n in RULE:
        for dtype in range(3):
            got = [next(it) for _ in range(n)]
            d, f, T, k = size[0], size[1], size[4], size[3]
            assert got[0][3:5] == [f // 32, T * k], size    # gate/up: a workgroup an f-block and pair
            assert (got[1][3] == d // 32 and got[1][5] == 1024) == (n == 2), size


def test_the_waves_of_a_pair(events):
    """Four waves a workgroup where there are more than two a CU and a wave of eight would have a ring of K at most."""
    it = iter([e for e in events if e[0] == "launch"][3 * sum(n for _, n in RULE):])
    for size, threads in WAVES:
        for dtype in range(3):
            assert [next(it) for _ in range(3)][0][5] == threads, size
