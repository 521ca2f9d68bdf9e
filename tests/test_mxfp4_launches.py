"""Which kernel a product takes, by the launches that a recording HIP runtime sees: each of the rule's borders."""
import pytest

from launch_recorder import record

MAIN = r"""
int main()
{
    static uint8_t none[256];
    std::printf("[");
    const int sizes[][5] = {SIZES};                       // M, N, K, groups (0: dense), swiglu
    for (auto& s : sizes) {
        moe::MxGemm g{};
        g.a_codes = g.a_scales = g.b_codes = g.b_scales = none, g.out = none;
        g.a_rows = g.M = s[0], g.N = s[1], g.K = s[2], g.row_div = 1, g.swiglu = s[4], g.out_stride = s[1], g.dtype = 1;
        g.G = s[3] ? s[3] : 1, g.bounds = s[3] ? reinterpret_cast<const int32_t*>(none) : nullptr;
        if (launch_mx_gemm(g, 0) != hipSuccess) return 1;
    }
    std::printf("]\n");
    return 0;
}
"""

# (M, N, K, groups, swiglu): rows of a tile, 32 for the few-row kernel
RULE = [((1, 4096, 4096, 0, 0), 32), ((64, 4096, 4096, 0, 0), 32), ((65, 4096, 4096, 0, 0), 64), ((512, 2048, 2048, 64, 0), 64),
        ((64, 8192, 4096, 0, 0), 64), ((512, 4096, 4096, 0, 0), 64), ((2048, 4096, 4096, 0, 0), 128),
        ((59 * 64, 2048, 2048, 64, 0), 64), ((60 * 64, 2048, 2048, 64, 0), 128), ((60 * 128, 768, 2048, 128, 1), 128),
        ((8192, 4096, 4096, 0, 0), 256), ((8192, 4096, 2816, 0, 0), 256), ((8192, 4096, 2784, 0, 0), 128), ((8192, 4096, 2048, 0, 0), 128),
        ((4096, 4096, 4096, 0, 0), 128), ((448 * 32, 2048, 4096, 32, 0), 256), ((447 * 32, 2048, 4096, 32, 0), 128)]


@pytest.fixture(scope="module")
def events(tmp_path_factory):
    main = MAIN.replace("SIZES", ", ".join("{%d, %d, %d, %d, %d}" % s for s, _ in RULE))
    return record(tmp_path_factory.mktemp("launches"), "moe_mx.h", "moe_mx.hip", main)


def test_the_rule_of_the_shapes(events):
    launches = [e for e in events if e[0] == "launch"]
    assert len(launches) == len(RULE)
    for (size, rows), (_, _, lds, _, gy, threads) in zip(RULE, launches):
        if rows == 32:
            assert (threads, lds, gy) == (512, 0, -(-size[1] // 32)), size
        else:                                             # two stages of (rows + columns of B) 128-byte rows, and the scales
            data = 2 * 128 * (rows + max(rows, 128))
            assert threads == 256 and data < lds < data * 1.3 + 8192, (size, lds)


def test_every_launch_is_within_its_kernels_limit(events):
    limit = {}
    for kind, f, v, *_ in events:
        if kind == "limit":
            assert limit.setdefault(f, v) == v and v <= 160 << 10
        else:
            assert v <= limit.get(f, 0)
