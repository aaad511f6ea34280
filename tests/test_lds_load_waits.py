"""The assembly of the kernels keeps the wait states that a buffer load needs
and that the compiler does not insert inside an asm block: one between the write
of M0 and a load to LDS, five between a vector instruction that writes a scalar
register and a memory instruction that reads it.  Every path of up to five
instructions back from each memory instruction is followed, through branches.
No GPU is needed: the sources are compiled to text."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from test_host_sanitizers import CSRC, _hipcc

SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith(".hip") and "lds_load16" in open(os.path.join(CSRC, f)).read())
VECTOR_WRITES_TWO = ("v_add_co", "v_sub_co", "v_subrev_co", "v_addc_co", "v_subb_co", "v_div_scale", "v_mad_u64", "v_mad_i64")


def scalars(operand):
    """The scalar registers of one operand."""
    m = re.fullmatch(r"s(\d+)", operand) or re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[m.lastindex]) + 1))
    return {"vcc"} if operand.startswith("vcc") else set()


class Instruction:
    def __init__(self, text):
        self.op, _, rest = text.replace("\t", " ").partition(" ")
        args = [a.strip() for a in re.split(r",(?![^\[]*\])", rest)]
        words = set(rest.replace(",", " ").split())
        self.text = text
        self.states = int(args[0], 0) + 1 if self.op == "s_nop" else 1
        self.memory = self.op.startswith(("buffer_", "global_", "flat_", "scratch_"))
        self.to_lds = self.memory and "lds" in words
        self.reads = set().union(*(scalars(w) for a in args for w in a.split())) if self.memory else set()
        self.writes = set()
        if self.op.startswith("v_"):
            self.writes = scalars(args[0])
            if self.op.startswith(VECTOR_WRITES_TWO):
                self.writes |= scalars(args[1])
        self.m0 = self.op.startswith("s_") and args[0] == "m0"
        self.to = args[0] if self.op.startswith(("s_branch", "s_cbranch")) else None
        self.ends = self.op in ("s_branch", "s_endpgm", "s_setpc_b64")


def faults(assembly):
    """Loads that come too early, as (number, load, the instruction they wait for)."""
    code, before, labels, falls = [], [], {}, None
    for line in assembly.splitlines():
        text = line.split(";")[0].split("//")[0].strip()
        m = re.fullmatch(r"([.\w$]+):", text)
        if m:
            labels[m[1]] = len(code)
            continue
        if not text or text.startswith("."):
            continue
        before.append([] if falls is None else [falls])
        code.append(Instruction(text))
        falls = None if code[-1].ends else len(code) - 1
    for i, x in enumerate(code):
        if x.to in labels and labels[x.to] < len(code):
            before[labels[x.to]].append(i)
    found = []
    for i, x in enumerate(code):
        if not x.memory:
            continue
        todo = [(p, 0) for p in before[i]]
        while todo:
            at, states = todo.pop()
            y = code[at]
            if y.writes & x.reads or (y.m0 and x.to_lds and states < 1):
                found.append((i, x.text, y.text))
            if states + y.states < 5:
                todo += [(p, states + y.states) for p in before[at]]
    return found


@pytest.mark.parametrize("text,count", [
    ("s_mov_b32 m0, s1\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds", 1),
    ("s_mov_b32 m0, s1\n s_nop 0\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds", 0),
    ("v_readlane_b32 s6, v1, 3\n s_mov_b32 m0, s1\n s_nop 2\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds", 1),
    ("v_readlane_b32 s6, v1, 3\n s_mov_b32 m0, s1\n s_nop 3\n buffer_load_dwordx4 v1, s[4:7], 0 offen lds", 0),
    ("v_readlane_b32 s8, v1, 3\n buffer_load_dwordx4 v1, v2, s[4:7], 0 offen", 0),
    ("v_cmp_eq_u32 s[0:1], v0, v1\n s_branch .L1\n.L0:\n s_nop 1\n.L1:\n global_load_dword v1, v0, s[0:1]", 1),
    ("v_cmp_eq_u32 s[0:1], v0, v1\n s_branch .L1\n.L0:\n s_nop 1\n.L1:\n global_load_dword v1, v0, s[2:3]", 0),
])
def test_the_check_itself(text, count):
    assert len(faults(text)) == count


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    from sparse_int4_gemm_amd import build
    out = tmp_path_factory.mktemp("asm")

    def compile_one(f):
        to = str(out / (f + ".s"))
        res = subprocess.run([hipcc, *build.COMMON_FLAGS, *build.FILE_FLAGS.get(f, []), "--offload-device-only", "-S",
                              os.path.join(CSRC, f), "-o", to], capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-4000:]
        return open(to).read()

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        return dict(zip(SOURCES, ex.map(compile_one, SOURCES)))


@pytest.mark.parametrize("source", SOURCES)
def test_loads_wait_for_what_they_read(assembly, source):
    assert "offen lds" in assembly[source]
    found = faults(assembly[source])
    assert not found, f"{len(found)} loads too early, the first: {found[0][1]!r} after {found[0][2]!r}"
