"""The prompt kernel's TMEM plan, shared-memory layout and registers, read from its source and checked on the CPU."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_attention_video_smooth_gb300", "csrc")


def _constants():
    env = {"kBlk": 128, "kD": 128}
    text = open(os.path.join(SRC, "vca_prompt.cu")).read()
    for m in re.finditer(r"^constexpr\s+(?:int|uint32_t)\s+([^;]*);", text, flags=re.M):
        for part in m.group(1).split(","):
            name, _, expr = part.partition("=")
            env[name.strip()] = int(eval(expr.replace("/", "//"), {"__builtins__": {}}, dict(env)))
    return env, text


def test_tmem_holds_both_tiles_scores_and_outputs():
    c, _ = _constants()
    spans = sorted([(c["kTmemS"] + 128 * t, c["kTmemS"] + 128 * (t + 1)) for t in range(c["kTiles"])] +
                   [(c["kTmemO"] + 128 * t, c["kTmemO"] + 128 * (t + 1)) for t in range(c["kTiles"])])
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])) and spans[-1][1] <= c["kTmemCols"] <= 512


def test_shared_memory():
    c, _ = _constants()
    assert c["kOffQ"] % 1024 == 0 and c["kOffKV"] % 1024 == 0 and c["kBlock"] % 1024 == 0      # the 128-byte swizzle's atoms
    assert c["kOffKV"] - c["kOffQ"] == c["kTiles"] * c["kBlock"] and c["kOffStat"] - c["kOffKV"] == c["kStages"] * c["kBlock"]
    assert c["kOffSort"] - c["kOffStat"] == 2 * c["kTiles"] * 2 * 128 * 4
    assert c["kOffBar"] - c["kOffSort"] == 3 * 4 * c["kSortable"] and c["kOffBar"] % 8 == 0
    # full, empty, raw; q_full, q_free, s_full, p_full in halves, o_full, o_free; w_full, w_free; drain
    used = 3 * c["kStages"] + 7 * c["kTiles"] + 2 * c["kWorks"] + 1
    assert used <= c["kNumBars"] and c["kOffWork"] >= c["kOffBar"] + 8 * c["kNumBars"] and c["kOffWork"] % 16 == 0
    assert c["kOffMisc"] == c["kOffWork"] + 16 * c["kWorks"] and c["kSmem"] <= 232448
    assert c["kStages"] & (c["kStages"] - 1) == 0      # copies are counted modulo 2^32


def test_registers_add_up():
    """What the four warpgroups ask for is no more than the block was launched with."""
    c, text = _constants()
    asked = [int(n) for n in re.findall(r"setmaxnreg\.\w+\.sync\.aligned\.u32 (\d+)", text)]
    assert len(asked) == 3 and c["kThreads"] == 512 and all(n % 8 == 0 for n in asked)
    at_launch = 65536 // c["kThreads"]
    other, softmax, out = asked
    assert 128 * (other + 2 * softmax + out) <= 512 * at_launch
