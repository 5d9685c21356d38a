"""The wait states between an MFMA and the first instruction that touches its result, in the
assembly that the build's flags give.  The hardware does not interlock them and the compiler
inserts them, but it has left them out where a result was first read behind a branch; values
then come out wrong, without an error and not in every run.  So every path is followed."""
import re
import subprocess

import pytest

from block_scaled_fp8_bsgemm_amd import _build

# Wait states until a vector instruction may touch the result: the passes (4 cycles each), and
# 4; both forms of the f8f6f4 product take 8 passes, the bf16 one 4.
WAITS = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x128_f8f6f4": 12, "v_mfma_scale_f32_16x16x128_f8f6f4": 12}
SOURCES = ("gemm.hip", "moe.hip", "lora.hip")


def registers(text):
    out = set()
    for m in re.finditer(r"(?<![a-z0-9_])v(?:\[(\d+):(\d+)\]|(\d+))", text):
        lo, hi = (int(m[1]), int(m[2])) if m[1] else (int(m[3]), int(m[3]))
        out.update(range(lo, hi + 1))
    return out


def functions(asm):
    """name -> (instructions, label -> index) of each function's code."""
    out, at = {}, None
    for line in asm.splitlines():
        line = line.split(";")[0].rstrip()
        if m := re.match(r"(_Z\w+):", line):
            at = out[m[1]] = ([], {})
        elif at is None:
            continue
        elif line.startswith("\t.end_amdhsa"):
            at = None
        elif m := re.match(r"(\.LBB\S+):", line):
            at[1][m[1]] = len(at[0])
        elif re.match(r"\t[a-z]", line):
            at[0].append(line.split(None, 1) if len(line.split(None, 1)) == 2 else [line.strip(), ""])
    return out


def short_waits(code, labels):
    """(MFMA, instruction, wait states between) wherever those are too few."""
    found = []
    for i, (op, args) in enumerate(code):
        if not op.startswith(("v_mfma", "v_smfmac")):
            continue
        need, result = WAITS[op], registers(args.split(",")[0])
        best, todo = {}, [(i + 1, 0)]
        while todo:
            j, waited = todo.pop()
            if j >= len(code) or waited >= need or best.get(j, need) <= waited:
                continue
            best[j] = waited
            o, a = code[j]
            if o.startswith("v_mfma"):
                d, x, y = (registers(p) for p in a.split(",")[:3])
                if (x | y) & result:     # as an operand; accumulating onto it has its own, shorter wait
                    found.append((op + " " + args, o + " " + a, waited))
                if d >= result:
                    continue
            elif o.startswith(("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")) and registers(a) & result:
                found.append((op + " " + args, o + " " + a, waited))
                continue
            if o == "s_endpgm":
                continue
            if o.startswith(("s_branch", "s_cbranch")):
                todo.append((labels[a.strip()], waited + 1))
            if o != "s_branch":
                todo.append((j + 1, waited + (int(a, 0) + 1 if o == "s_nop" else 1)))
    return found


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    out = tmp_path_factory.mktemp("asm")
    flags = [f for f in _build.HIPCC_FLAGS if f != "-shared"]
    runs = []
    for s in SOURCES:
        cmd = [_build.hipcc(), *flags, "-w", "--cuda-device-only", "-S", "-I", _build.INCLUDE, "-I", _build.CSRC,
               f"{_build.CSRC}/{s}", "-o", str(out / s)]
        runs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT))
    for r in runs:
        text = r.communicate()[0]
        assert r.returncode == 0, text.decode()
    return {s: (out / s).read_text() for s in SOURCES}


@pytest.mark.parametrize("source", SOURCES)
def test_no_short_waits(assembly, source):
    kernels = functions(assembly[source])
    products = 0
    for name, (code, labels) in kernels.items():
        products += sum(op.startswith("v_mfma") for op, _ in code)
        assert not short_waits(code, labels), (name, short_waits(code, labels)[:3])
    assert products > 100      # the search found the code


SNIPPET = """
_Z1kv:
\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0
\ts_nop 3
\ts_cbranch_scc1 .LBB0_2
\ts_nop {nop}
.LBB0_2:
\t{use}
\ts_endpgm
\t.end_amdhsa_kernel
"""


@pytest.mark.parametrize("nop,use,bad", [
    (7, "v_fma_f32 v4, v2, v5, v6", [5]),                       # on the branch's way
    (7, "v_fma_f32 v4, v7, v5, v6", []),
    (7, "v_mov_b32_e32 v3, 0", [5]),
    (7, "ds_write_b128 v20, v[0:3]", [5]),
    (7, "s_nop 2\n\tv_fma_f32 v4, v2, v5, v6", []),
    (7, "v_mfma_f32_16x16x32_bf16 v[16:19], v[0:3], v[12:15], 0", [5]),
    (7, "v_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[12:15], v[0:3]", []),
])
def test_the_search_itself(nop, use, bad):
    code, labels = functions(SNIPPET.format(nop=nop, use=use))["_Z1kv"]
    assert [w for _, _, w in short_waits(code, labels)] == bad
