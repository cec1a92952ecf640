"""CPU test of the built library's machine code: the vector unit touches no register of a matrix instruction's result before
the result is there.  The hardware does not wait; the compiler counts the states, and has counted them wrongly where one of two
ways to a place passes a branch by, which gave wrong results now and then.  Every way through each kernel is followed here.

A 16x16x32 product of 16 bits takes 4 passes; its result may be read, or its registers written, by the vector unit, and read by
a store, 8 states after it was issued.  An instruction is a state, s_nop n is n + 1.  Another product that adds to the same
registers waits by itself."""
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STATES = 8
LINE = re.compile(r"^\t(\S+)\s*(.*?)\s*// [0-9A-F]+:")
LABEL = re.compile(r"^[0-9a-f]+ <(.+)>:")
REGISTER = re.compile(r"\b([va])(?:(\d+)|\[(\d+):(\d+)\])(?![\w\[])")


def registers(text):
    out = set()
    for kind, one, first, last in REGISTER.findall(text):
        out |= {kind + one} if one else {f"{kind}{i}" for i in range(int(first), int(last) + 1)}
    return out


def operands(text):
    return [x.strip() for x in re.split(r",(?![^\[]*\])", text)]


def kernels(listing):
    """name -> (instructions, label -> index) of a disassembly."""
    found, code, labels = {}, [], {}
    for line in listing.splitlines():
        label, ins = LABEL.match(line), LINE.match(line)
        if label and re.fullmatch(r"L\d+", label.group(1)):
            labels[label.group(1)] = len(code)
        elif label:
            code, labels = [], {}
            found[label.group(1)] = code, labels
        elif ins:
            code.append((ins.group(1), operands(ins.group(2))))
    return found


def touches(op, args, result):
    """Whether the vector unit reads or writes, or a store or an address reads, a register of `result`."""
    if op.startswith("v_"):
        return bool(registers(",".join(args)) & result)
    if op.startswith(("global_", "flat_", "scratch_", "buffer_", "ds_")):
        loads = "load" in op or "read" in op
        to_lds = "lds" in op
        return bool(registers(",".join(args[1:] if loads and not to_lds else args)) & result)
    return False


def early(code, labels):
    """(product, toucher, states between) of each result touched too early on some way, and how many products there are."""
    def after(k):
        op, args = code[k]
        ways = [] if op in ("s_endpgm", "s_branch") or k + 1 == len(code) else [k + 1]
        return ways + [labels[args[0]]] if op.startswith(("s_cbranch", "s_branch")) else ways

    bad, products = [], 0
    for k, (op, args) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        products += 1
        assert op in ("v_mfma_f32_16x16x32_bf16", "v_mfma_f32_16x16x32_f16"), f"{op}: its states are not known here"
        to, result = args[0], registers(args[0])
        best, ways = {}, [(n, 0) for n in after(k)]
        while ways:
            at, passed = ways.pop()
            if passed >= STATES or best.get(at, STATES) <= passed:
                continue
            best[at] = passed
            other, theirs = code[at]
            if other.startswith("v_mfma"):
                if registers(",".join(theirs[1:3])) & result or (theirs[3] != to and registers(theirs[3]) & result):
                    bad.append(((op, args), (other, theirs), passed))
                elif theirs[0] == to:
                    continue   # the same registers: that one's result counts from here on
            elif touches(other, theirs, result):
                bad.append(((op, args), (other, theirs), passed))
                continue
            states = int(theirs[0], 0) + 1 if other == "s_nop" else 1
            ways += [(n, passed + states) for n in after(at)]
    return bad, products


def lines(*code):
    return "0000000000001000 <k>:\n" + "".join(c + "\n" if c.endswith(">:") else f"\t{c} // 00000000{i:04X}: 00\n" for i, c in enumerate(code))


def test_the_count_follows_every_way():
    product = "v_mfma_f32_16x16x32_f16 v[0:3], v[4:7], v[8:11], 0"
    past = [product, "s_cbranch_vccnz L0", "s_nop 7", "0000000000001010 <L0>:", "v_add_f32_e32 v20, v1, v20", "s_endpgm"]
    bad, products = early(*kernels(lines(*past))["k"])
    assert products == 1 and [b[2] for b in bad] == [1]   # the branch alone is between them
    assert early(*kernels(lines(product, "s_nop 7", *past[1:]))["k"])[0] == []
    assert early(*kernels(lines(product, "s_nop 6", "s_endpgm"))["k"]) == ([], 1)
    short = [product, "s_nop 6", "global_store_dwordx4 v[30:31], v[0:3], off", "s_endpgm"]
    assert [b[2] for b in early(*kernels(lines(*short))["k"])[0]] == [7]
    again = [product, "v_mfma_f32_16x16x32_f16 v[0:3], v[4:7], v[8:11], v[0:3]", "s_nop 7", "v_mov_b32_e32 v0, 0", "s_endpgm"]
    assert early(*kernels(lines(*again))["k"]) == ([], 2)
    operand = [product, "v_mfma_f32_16x16x32_f16 v[12:15], v[0:3], v[8:11], 0", "s_endpgm"]
    assert [b[2] for b in early(*kernels(lines(*operand))["k"])[0]] == [0]


def test_no_result_of_the_built_kernels_is_touched_early(tmp_path):
    objdump = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump to list the kernels with")
    lib = os.path.join(ROOT, "copy_reduce_amd", "libtb.so")
    assert os.path.exists(lib), "build first (python -c 'import __graft_entry__ as g; g.build()')"
    shutil.copy(lib, tmp_path / "lib.so")
    subprocess.run([objdump, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    checked = {}
    for image in sorted(glob.glob(str(tmp_path / "*gfx950*"))):
        listing = subprocess.run([objdump, "-d", "--symbolize-operands", image], check=True, capture_output=True, text=True).stdout
        for name, (code, labels) in kernels(listing).items():
            if "v_mfma" not in listing:
                break
            bad, products = early(code, labels)
            assert not bad, f"{name}: {len(bad)} results touched early, the first: {bad[0]}"
            if products:
                checked[name] = products
    shared = [n for n in checked if "tree_attention_shared_kernel" in n]
    few = [n for n in checked if "tree_attention_kernel" in n]
    # 2 types, 4 head sizes; few rows: 3 forms; many: of 2, 4 and 8 waves with rows (256 elements: 4 and 8), 3 forms
    assert len(few) == 24 and len(shared) == 66, (len(few), len(shared))
