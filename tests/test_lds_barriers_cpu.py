"""The built gfx950 code: no wave reaches a barrier with LDS writes of its own still under way.

s_barrier waits for no memory operation, so a wave that passes it could read what another one's write has not yet
replaced.  Every path of every kernel in the library is followed from its start: a write to LDS is under way until an
s_waitcnt lgkmcnt(0)."""
import re
import shutil
import struct
import subprocess

import pytest

import fp8_w8a8_quantized_quantize_amd as fp8
from fp8_w8a8_quantized_quantize_amd import _build

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
LINE = re.compile(r"^\t(\S+)(.*?)// ([0-9A-F]+):")


def code_objects():
    """The gfx950 code objects of the library, one per source with kernels."""
    data = open(_build.LIB, "rb").read()
    at, out = data.find(MAGIC), []
    while at >= 0:
        n, = struct.unpack_from("<Q", data, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + length] and size:
                out.append(data[at + off:at + off + size])
            p += 24 + length
        at = data.find(MAGIC, at + 1)
    return out


def kernels(text):
    """(name, [(address, mnemonic, operands)]) of each function of a disassembly."""
    name, body = None, []
    for line in text.splitlines():
        head = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
        if head:
            if name:
                yield name, body
            name, body = head.group(1), []
            continue
        m = LINE.match(line)
        if m:
            body.append((int(m.group(3), 16), m.group(1), line[m.end(1):]))
    if name:
        yield name, body


def barriers_with_writes(body):
    """(barriers, addresses of those that some path reaches with LDS writes under way)."""
    index = {a: i for i, (a, _, _) in enumerate(body)}
    base = body[0][0]
    seen, bad, barriers = [set() for _ in body], set(), set()
    todo = [(0, False)]
    while todo:
        i, pending = todo.pop()
        while i < len(body) and pending not in seen[i]:
            seen[i].add(pending)
            addr, op, rest = body[i]
            if op.startswith("ds_") and re.match(r"ds_(write|add|sub|inc|dec|min|max|and|or|xor|cmpst|wrxchg)", op):
                pending = True
            elif op == "s_waitcnt" and "lgkmcnt(0)" in rest:
                pending = False
            elif op == "s_barrier":
                barriers.add(addr)
                if pending:
                    bad.add(addr)
            elif op == "s_endpgm":
                break
            if op.startswith(("s_cbranch", "s_branch")):
                target = re.search(r"<\S+?(?:\+0x([0-9a-f]+))?>\s*$", rest)
                assert target, f"{op}{rest}"
                j = index[base + int(target.group(1) or "0", 16)]
                if op == "s_branch":
                    i = j
                    continue
                todo.append((j, pending))
            i += 1
    return barriers, bad


def stores_before_a_barrier(body):
    """Global stores that some path reaches without a barrier before them."""
    index, base = {a: i for i, (a, _, _) in enumerate(body)}, body[0][0]
    seen, bad, todo = set(), [], [0]
    while todo:
        i = todo.pop()
        while i < len(body) and i not in seen:
            seen.add(i)
            addr, op, rest = body[i]
            if op.startswith("global_store"):
                bad.append(addr)
            if op in ("s_barrier", "s_endpgm"):
                break
            if op.startswith(("s_cbranch", "s_branch")):
                j = index[base + int(re.search(r"<\S+?(?:\+0x([0-9a-f]+))?>\s*$", rest).group(1) or "0", 16)]
                if op == "s_branch":
                    i = j
                    continue
                todo.append(j)
            i += 1
    return bad


@pytest.fixture(scope="module")
def functions():
    fp8.lib()
    if not shutil.which(OBJDUMP):
        pytest.skip("no disassembler")
    out = []
    for obj in code_objects():
        text = subprocess.run([OBJDUMP, "-d", "-"], input=obj, capture_output=True, check=True).stdout.decode()
        out += list(kernels(text))
    return out


def test_no_lds_write_under_way_at_a_barrier(functions):
    found, bad = 0, {}
    for name, body in functions:
        barriers, wrong = barriers_with_writes(body)
        found += len(barriers)
        if wrong:
            bad[name] = [hex(a) for a in sorted(wrong)]
    assert found > 100, "barriers in the disassembly"
    assert not bad, f"{len(bad)} kernels: {dict(list(bad.items())[:4])}"


def test_products_store_behind_a_barrier(functions):
    """A product's outputs need scales that other waves put into LDS, so no path to a store is without a barrier -- that
    of an empty K, which no step of the K loop lies on, included."""
    products = [(name, body) for name, body in functions if "gemm_mfma_kernel" in name]
    assert len(products) > 20
    bad = {name: [hex(a) for a in at] for name, at in ((n, stores_before_a_barrier(b)) for n, b in products) if at}
    assert not bad, f"{len(bad)} kernels: {dict(list(bad.items())[:4])}"


def test_the_check_itself():
    """Writes before a branch, in a loop and behind a wait."""
    def body(*ops):
        return [(4 * i, *(o + (("",) if len(o) == 1 else ()))) for i, o in enumerate(ops)]

    end, wait, bar = ("s_endpgm",), ("s_waitcnt", " lgkmcnt(0)"), ("s_barrier",)
    assert barriers_with_writes(body(("ds_write_b128",), bar, end)) == ({4}, {4})
    assert barriers_with_writes(body(("ds_write_b128",), wait, bar, end)) == ({8}, set())
    assert barriers_with_writes(body(("ds_add_u32",), ("s_cbranch_scc0", " 1  <f+0xc>"), wait, bar, end)) == ({12}, {12})
    assert barriers_with_writes(body(bar, ("ds_write_b32",), ("s_cbranch_scc0", " 65533  <f>"), end)) == ({0}, {0})
    assert barriers_with_writes(body(bar, ("ds_read_b32",), ("s_cbranch_scc0", " 65533  <f>"), end)) == ({0}, set())
