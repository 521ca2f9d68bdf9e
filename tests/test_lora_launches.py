"""How many launches the adapters of a few rows take, by a recording HIP runtime, at the borders of the rule."""
from launch_recorder import record
from test_experts16_abi import LORA

# M, K, N, r, fp32 base and out: launches
RULE = [((1, 4096, 4096, 32, 0), 1), ((1, 4096, 4096, 40, 0), 2), ((1, 4096, 4096, 16, 1), 1), ((1, 2048, 4096, 24, 1), 1), ((1, 2048, 4096, 32, 1), 2),
        ((1, 4096, 4096, 24, 1), 2), ((1, 4096, 4095, 24, 1), 1), ((16, 1184, 2048, 32, 1), 1), ((16, 2048, 2048, 32, 1), 2), ((16, 2048, 2048, 32, 0), 1),
        ((48, 1184, 2051, 24, 1), 1)]


def test_one_launch_or_two(tmp_path):
    main = LORA.replace("SIZES", ", ".join("{%d, %d, %d, %d, %d}" % s for s, _ in RULE))
    events = [e for e in record(tmp_path, "moe_lora.h", "moe_lora.hip", main) if e[0] == "launch"]
    got = []
    for e in events:                                      # one launch: 512 threads; two: 256, then 256
        if e[5] == 512:
            got.append(1)
        elif got and got[-1] == 0:
            got[-1] = 2
        else:
            got.append(0)
    assert got == [n for _, n in RULE]
