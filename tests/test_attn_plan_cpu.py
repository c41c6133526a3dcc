"""How the attention calls are divided into workgroups, on the host: grids that the runtime takes (less than 2^32
threads along an axis) at every size the entry points accept, whatever the launch hints say, and slots that hold every
column tile of a ragged batch."""
import bisect
import ctypes
import os
import random
import subprocess
import tempfile

import pytest

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None
THREADS, MAX_ATTN = 256, 1 << 30


def lib():
    global _lib
    if _lib is None:
        out = os.path.join(tempfile.mkdtemp(prefix="fp8planpin_"), "libplan_pin.so")
        subprocess.run(["g++", "-O2", "-fPIC", "-shared", "-std=c++17", "-Wall", "-Werror",
                        os.path.join(_HERE, "pins", "attn_plan_pin.cpp"), "-o", out], check=True)
        _lib = ctypes.CDLL(out)
    return _lib


def plan(fn, *args):
    out = (ctypes.c_int64 * 4)()
    getattr(lib(), fn)(*[ctypes.c_int64(int(a)) for a in args], out)
    return list(out)


def launches(units):
    """A kernel's workgroups, in launches that the runtime takes."""
    assert 1 <= units < 1 << 31
    n, total, largest = plan("pin_launches", units)[:3]
    assert total == units and largest * THREADS < 1 << 32
    assert n == -(-units // (((1 << 32) - 1) // THREADS))
    return n


def check(B, rows, Hq, Hkv, D, max_q, max_len, all_len, decode):
    """Every launch that the call may make."""
    what = (B, rows, Hq, Hkv, D, max_q, max_len, all_len, decode)
    units, y, shares = plan("pin_stream", B, rows, Hq, Hkv, D, max_q, max_len, all_len)[:3]
    assert 1 <= y <= 65535 and (y == 1 or not shares), what
    launches(units)
    units, slots, splits = plan("pin_tiled", B, rows, Hq, Hkv, D, decode, max_q, max_len)[:3]
    assert units == slots * Hkv * splits, what
    launches(units)
    for heads, q, typical in ((B * Hq, max_q, max_q), (B * Hq, max_q, -(-rows // B)), (Hq, rows, rows)):
        units, per, spread = plan("pin_join", heads, D, q, typical)[:3]
        launches(units)
        assert 1 <= per <= q and units * (THREADS // (D // 4)) // spread >= heads * per, what
    return slots * Hkv


@pytest.mark.parametrize("T,B", [(65536, 512), (131072, 256), (32768, 1024)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_ragged_batches_without_a_hint(T, B, D):
    """An unknown max_q counts as T; the launch is as large as the batch all the same."""
    tiles = check(B, T, 64, 8, D, T, 4096, 4096, False)
    assert tiles <= (T * 8 // 128 + B) * 8


@pytest.mark.parametrize("B,rows,Hq,Hkv,max_q,all_len", [
    (1 << 26, 1 << 26, 1, 1, 1, 1), (1 << 26, 1 << 26, 1, 1, 1 << 26, 1 << 30), (1 << 25, 1 << 25, 2, 1, 1, 700),
    (1 << 25, 1 << 25, 2, 2, 1, 1 << 30), (1024, 1 << 14, 1 << 16, 65535 // 3, 1 << 14, 1 << 20), (1, 1 << 30, 1, 1, 1 << 30, 1 << 30),
    (1 << 10, 1 << 14, 1 << 16, 1 << 15, 1, 64), (1 << 26, 1, 1, 1, 1, 1 << 30), (1, 1, 1 << 22, 1, 1, 1 << 30)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_largest_sizes(B, rows, Hq, Hkv, max_q, all_len, D):
    Hq = Hq // Hkv * Hkv
    for max_len in (1, min(700, all_len), all_len):
        check(B, rows, Hq, Hkv, D, max_q, max_len, all_len, False)
        check(B, B, Hq, Hkv, D, 1, max_len, all_len, True)


def test_any_accepted_size():
    rng = random.Random(5)

    def upto(n):
        return min(n, 1 << rng.randint(0, max(0, n.bit_length() - 1))) + rng.randint(0, 3)

    for _ in range(20000):
        D = rng.choice([64, 128, 256])
        B = min(upto(1 << 26), 1 << 26)
        Hq = max(1, min(upto((1 << 26) // B), (1 << 26) // B, MAX_ATTN // D))
        Hkv = rng.choice([d for d in range(1, min(Hq, 65535) + 1) if Hq % d == 0][:40])
        decode = rng.random() < 0.4
        rows = B if decode else max(1, min(upto(MAX_ATTN // Hq), MAX_ATTN // Hq))
        all_len = min(upto(MAX_ATTN), MAX_ATTN)
        max_q = 1 if decode else rng.choice([rows, min(rows, upto(rows)), 1])
        check(B, rows, Hq, Hkv, D, max_q, min(all_len, upto(all_len)), all_len, decode)


@pytest.mark.parametrize("Hkv,most", [(1, 90), (400, 90), (2, 1500)])
def test_slots_hold_every_column_tile(Hkv, most):
    """The kernel's arithmetic: a first tile for every sequence where the hint, right or wrong, says that one will do, and
    all others end to end; or the last sequence that starts at or before a slot, when b starts at
    floor(cu[b] * group / 128) + b."""
    rng = random.Random(7)
    forms = set()
    for _ in range(300 if most < 100 else 12):
        B, group = rng.randint(1, most), rng.choice([1, 2, 3, 8, 16, 127, 128, 129, 300])
        new = [rng.choice([0, 0, 1, 2, 16, rng.randint(0, 40), rng.randint(0, 700)]) for _ in range(B)]
        if rng.random() < 0.3:
            new = [rng.randint(max(0, new[0] - 2), new[0]) for _ in range(B)]
        cu = [rng.choice([0, 0, 5])]
        for n in new:
            cu.append(cu[-1] + n)
        rows = max(cu[-1] + rng.choice([0, 0, 9]), 1)
        hint = max(1, min(rows, rng.choice([rows, max(new), max(new), 1, 20])))
        slots, _, form = plan("pin_tiled", B, rows, group * Hkv, Hkv, 128, False, hint, 4096)[1:]
        exact, each = form >= 1000, form % 1000
        forms.add((exact, each))
        tiles = [-(-n * group // 128) for n in new]
        others = [max(t - each, 0) for t in tiles]
        starts = [c * group // 128 + b for b, c in enumerate(cu[:-1])]
        if exact:
            starts = [0]
            for t in others:
                starts.append(starts[-1] + t)
        seen = [(slot % B, each - 1 - slot // B) for slot in range(B * each)]
        seen = [(b, ct) for b, ct in seen if ct < tiles[b]]
        for slot in range(slots - B * each):
            slot = slot if exact else slots - 1 - slot
            b = bisect.bisect_right(starts, slot, 0, B) - 1
            if b >= 0 and slot - starts[b] < others[b]:
                seen.append((b, each + slot - starts[b]))
        assert sorted(seen) == [(b, ct) for b in range(B) for ct in range(tiles[b])], (new, group, cu[0], hint)
    assert len(forms) > 1


def test_launches_past_a_grid():
    most = ((1 << 32) - 1) // THREADS
    assert [launches(n) for n in (1, most, most + 1, 2 * most, 2 * most + 1)] == [1, 1, 2, 2, 3]


@pytest.mark.parametrize("B,new,Hq,Hkv", [(32, 4, 32, 8), (256, 3, 64, 8), (64, 1, 64, 8), (1024, 2, 64, 8), (3, 2, 8, 2)])
@pytest.mark.parametrize("max_len", [500, 1000, 30000])
def test_few_new_tokens_without_a_hint(B, new, Hq, Hkv, max_len):
    """Drafted tokens whose bound is not told (all T rows) take the streaming form by their mean, and workgroups of the
    order of what there is to do, not B times T."""
    T = B * new
    assert plan("pin_form", Hq, Hkv, 128, new, 0)[0] == 0
    tiles = B + T * (Hq // Hkv) // 16
    units, y, shares = plan("pin_stream", B, T, Hq, Hkv, 128, T, max_len, 40000)[:3]
    assert units * y <= max(4096, 4 * tiles * Hkv)
    units, per, spread = plan("pin_join", B * Hq, 128, T, new)[:3]
    assert units <= max(16384, T * Hq)


def test_whole_prompts_without_a_hint():
    assert plan("pin_form", 64, 8, 128, 8192, 0)[0] == 1
    assert plan("pin_form", 8, 8, 64, 256, 1)[0] == 1
