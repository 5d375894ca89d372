"""The assembly of the absorbed attention's kernels (CPU only): their sums lie in
registers that products written as assembly add to, where the compiler puts no
waits, so no path may touch them within the 19 wait states that a product of 16
passes needs, except the next product of the same sums."""

import re
import subprocess

import pytest

from fp8_blockwise_weight_amd import build as fb

WAIT = 19
SOURCE = """#include "fp8bq.h"
#include "../fp8_blockwise_weight_amd/csrc/kernels.hpp"
#include "../fp8_blockwise_weight_amd/csrc/latent_kernels.hpp"
"""


def registers(text):
    out = set()
    for kind, a, b, one in re.findall(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        out.update((kind, i) for i in (range(int(one), int(one) + 1) if one else range(int(a), int(b) + 1)))
    return frozenset(out)


def blocks_of(body):
    """Labels, and instructions (text, whether it is written as assembly)."""
    order, blocks, written = ["entry"], {"entry": []}, False
    for line in body.split("\n"):
        if "#ASMSTART" in line or "#ASMEND" in line:
            written = "#ASMSTART" in line
            continue
        code = line.split(";")[0].strip()
        label = re.match(r"(\.LBB\w+):", code)
        if label:
            order.append(label.group(1))
            blocks[order[-1]] = []
        elif code and not code.startswith("."):
            blocks[order[-1]].append((code, written))
    return order, blocks


def touched_early(body):
    """Instructions that touch sums too early, over every path; and how many
    products there are."""
    order, blocks = blocks_of(body)
    entry = {label: None for label in order}
    entry["entry"] = {}
    work, found, products = ["entry"], set(), set()
    while work:
        label = work.pop()
        state, after, falls = dict(entry[label]), [], True
        for i, (code, written) in enumerate(blocks[label]):
            op = code.split()[0]
            rest = code[len(op):]
            if op.startswith("v_mfma") and written:
                products.add((label, i))
                parts = re.findall(r"[va]\[\d+:\d+\]", rest)
                to = registers(parts[0])
                others = registers(" ".join(parts[1:3]))
                found.update((label, i, code) for p in state if p & others or (p & to and p != to))
                state = {p: n + 1 for p, n in state.items() if p != to and n + 1 < WAIT}
                state[to] = 0
            else:
                regs = registers(rest)
                found.update((label, i, code) for p in state if p & regs)
                step = int(rest) + 1 if op == "s_nop" else 1
                state = {p: n + step for p, n in state.items() if n + step < WAIT}
            if op.startswith("s_cbranch") or op == "s_branch":
                after.append((rest.strip(), dict(state)))
            if op in ("s_branch", "s_endpgm"):
                falls = False
                break
        if falls and order.index(label) + 1 < len(order):
            after.append((order[order.index(label) + 1], state))
        for to, s in after:
            known = entry[to]
            merged = dict(s) if known is None else {p: min(s.get(p, WAIT), known.get(p, WAIT)) for p in {**s, **known}}
            if merged != known:
                entry[to] = merged
                work.append(to)
    return found, len(products)


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    where = tmp_path_factory.mktemp("asm")
    src, out = where / "latent.hip", where / "latent.s"
    kernels = "".join(
        f"template __global__ void fp8bq::latent_attend<{n}, {w}>(LatentCache, KvBatch, LatentQuery);\n"
        for n in (256, 512) for w in (2, 4))
    text = SOURCE.replace("../", fb.ROOT + "/")
    src.write_text(text + "using namespace fp8bq;\n" + kernels)
    cmd = [c for c in fb.command(str(out)) if c not in ("-shared", "-fPIC", fb.SRC)]
    res = subprocess.run([cmd[0], "-S", "--cuda-device-only", *cmd[1:], str(src)], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-3000:]
    return out.read_text()


def test_sums_are_waited_for(asm):
    kernels = re.findall(r"^(_ZN5fp8bq13latent_attend\w+):(.*?)^\.Lfunc_end", asm, re.M | re.S)
    assert len(kernels) == 4
    for name, body in kernels:
        found, products = touched_early(body)
        assert products >= 8, name
        assert not found, (name, sorted(found)[:4])


def test_early_touches_are_seen():
    """The check itself, on paths with and without a wait."""
    product = "\t;;#ASMSTART\n\tv_mfma_scale_f32_32x32x64_f8f6f4 a[0:15], v[0:7], v[8:15], a[0:15], v1, v2\n\t;;#ASMEND\n"
    move, leave = "\tv_accvgpr_read_b32 v20, a3\n", "\ts_endpgm\n"
    wait = "\ts_nop 15\n\ts_nop 15\n"
    for body, bad in ((product + move + leave, 1), (product + wait + move + leave, 0), (product + product + leave, 0),
                      (product + "\ts_cbranch_scc1 .LBB0_2\n" + wait + ".LBB0_2:\n" + move + leave, 1),
                      (".LBB0_1:\n" + move + product + "\ts_cbranch_scc1 .LBB0_1\n" + leave, 1),
                      (".LBB0_1:\n" + move + product + wait + "\ts_cbranch_scc1 .LBB0_1\n" + leave, 0)):
        found, products = touched_early(body)
        assert (len(found), products) == (bad, body.count("v_mfma"))


# The kernels as they ship: in the library's own unit.

@pytest.fixture(scope="module")
def library_asm(tmp_path_factory):
    out = tmp_path_factory.mktemp("asm") / "library.s"
    cmd = [c for c in fb.command(str(out)) if c not in ("-shared", "-fPIC")]
    res = subprocess.run([cmd[0], "-S", "--cuda-device-only", *cmd[1:]], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-3000:]
    return out.read_text()


def bodies(text, kernel):
    return re.findall(rf"^(_ZN5fp8bq\d+{kernel}I\w+):(.*?)^\.Lfunc_end", text, re.M | re.S)


def test_sums_are_waited_for_in_the_library(library_asm):
    kernels = bodies(library_asm, "latent_attend")
    assert len(kernels) == 4
    for name, body in kernels:
        found, products = touched_early(body)
        assert products >= 8, name
        assert not found, (name, sorted(found)[:4])


def written_by_hand(body):
    """Instructions written as assembly."""
    _, blocks = blocks_of(body)
    return [code for block in blocks.values() for code, written in block if written]


def test_assembly_leaves_m0_to_the_compiler(library_asm):
    """Loads into LDS take their place from m0: as an operand, which the compiler
    sets and knows of.  An instruction that wrote it behind the compiler's back
    would change what the compiler's own uses of m0 read."""
    for kernel, count in (("latent_attend", 4), ("latent_prompt", 4)):
        kernels = bodies(library_asm, kernel)
        assert len(kernels) == count
        for name, body in kernels:
            codes = written_by_hand(body)
            assert any(code.startswith("global_load_lds") for code in codes), name
            assert not [code for code in codes if re.search(r"\bm0\b", code)], name
            assert re.search(r"^\ts_\w+ m0, ", body, re.M), name
