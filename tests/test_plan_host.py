"""How a call of tt_linear_loss is cut up (csrc/tt_plan.h), compiled for the host:
parts of contractions, chunks of rows, scratch."""
import ctypes
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
F32, F16, BF16 = range(3)


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "libplan_host.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "plan_host.cpp")])
    lib = ctypes.CDLL(so)
    lib.plan_host.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 6 + [ctypes.c_void_p]
    lib.plan_host_splits.argtypes = [ctypes.c_int, ctypes.c_int64]

    def call(n, vocab, dim, kind, pack_h=False, pack_w=False, dh=True, dw=True, dw_f32=False):
        """(rows of a chunk, parts of dhidden's contraction, of dweight's, bytes)"""
        out = (ctypes.c_int64 * 4)()
        lib.plan_host(n, vocab, dim, kind, pack_h, pack_w, dh, dw, dw_f32, out)
        return tuple(out)
    call.splits = lib.plan_host_splits
    lib.plan_host_patience.argtypes = [ctypes.c_void_p, ctypes.c_int]
    call.patience = lambda looks: lib.plan_host_patience((ctypes.c_uint64 * len(looks))(*looks), len(looks))
    return call


def sizes(count, seed):
    rng = random.Random(seed)
    for _ in range(count):
        vocab = rng.choice([300, 4352, 50257, 100256, 128256, 151936, 200256, 1 << 20, int(2 ** rng.uniform(0, 20))])
        yield int(2 ** rng.uniform(0, 24)), vocab, rng.choice([64, int(2 ** rng.uniform(0, 16))]), rng.choice([F32, F16, BF16])


def test_every_part_of_a_contraction_has_a_block(plan):
    """A part without one would be a tile that nothing is multiplied for, left with what its
    tensor memory held before: float, 151,936 tokens, 18,433 rows are chunks of 2304, two
    parts each, and a last one of a single row."""
    assert plan(18433, 151936, 64, F32, True, True)[:3] == (2304, 75, 2)
    short = 0
    for n, vocab, dim, kind in list(sizes(20000, 1)) + [(18433 + i, 151936, 64, F32) for i in range(66)]:
        chunk, split_h, split_w, _ = plan(n, vocab, dim, kind, kind == F32, kind == F32)
        last = n - (n - 1) // chunk * chunk
        for planned, k in ((split_h, vocab), (split_w, min(n, chunk)), (split_w, last)):
            if k == vocab and n <= (64 if kind == F32 else 4):
                continue                                   # (dhidden of few rows: parts of tokens, another kernel's)
            blocks, parts = (k + 63) // 64, plan.splits(planned, k)
            assert parts >= 1
            assert all(blocks * i // parts < blocks * (i + 1) // parts for i in range(parts)), (n, vocab, dim, kind, k)
            short += parts < planned
    assert short > 60                                      # (the last chunks of the sizes above)


def test_no_call_needs_more_scratch_than_is_asked_for(plan):
    """tt_linear_loss_workspace knows whether gradients are wanted, not which, and whether
    copies are, not of what: 143,337 rows of bf16, 7,471 tokens, a width of 7,504 and dhidden
    alone wanted more than both gradients."""
    cases = list(sizes(1000, 2)) + [(143337, 7471, 7504, BF16), (13513788, 44, 1832, BF16), (240000, 4352, 4416, BF16)]
    rng = random.Random(3)
    for _ in range(1000):                                  # widths above the vocabulary
        dim = int(2 ** rng.uniform(6, 16))
        cases.append((int(2 ** rng.uniform(10, 24)), rng.randrange(1, dim + 1), dim, rng.choice([F32, F16, BF16])))
    for n, vocab, dim, kind in cases:
        for pack in ((True,) if kind == F32 else (False, True)):
            packs = [(True, True)] if kind == F32 else [(True, True), (True, False), (False, True)] if pack else [(False, False)]
            alone = plan(n, vocab, dim, kind, pack, pack, False, False)
            assert all(plan(n, vocab, dim, kind, *p, False, False)[3] <= alone[3] for p in packs)
            for wide in {False, kind == F32}:
                most = plan(n, vocab, dim, kind, pack, pack, True, True, wide)
                for p in packs:
                    for dh, dw in ((True, True), (True, False), (False, True)):
                        for dhidden_alone in ((False, True) if not dw else (wide,)):  # (no dweight: its type is not looked at)
                            got = plan(n, vocab, dim, kind, *p, dh, dw, dhidden_alone)
                            assert got[0] == most[0] and got[3] <= most[3], (n, vocab, dim, kind, p, dh, dw)
            floats = plan(n, vocab, dim, kind, pack, pack, True, True, True)  # (16 bits into a float dweight)
            for p in packs:
                for dh, dw in ((True, True), (True, False), (False, True)):
                    assert plan(n, vocab, dim, kind, *p, dh, dw, True)[3] <= floats[3], (n, vocab, dim, kind, p, dh, dw)


def test_scratch_of_floats_with_gradients(plan):
    """What the header says of it: copies of 6 bytes a value, G of 2 GB at most or 256 rows, and
    sums of dhidden's parts of 2048 tokens, which nothing bounds but the sizes."""
    for n, vocab, dim in ((4096, 200256, 4096), (1024, 200256, 2112), (70, 1 << 20, 64), (3000, 4352, 1024)):
        rows, split_h, split_w, need = plan(n, vocab, dim, F32, True, True, True, True, True)
        g = (vocab + 63) // 64 * 64 * 6 * rows
        assert split_h >= (vocab + 2047) // 2048 and (g <= 2 << 30 or rows == 256)
        sums = 4 * dim * max(split_h * rows, split_w * vocab if split_w > 1 else 0)
        least = 6 * dim * (vocab + 2 * rows) + g + sums
        assert least <= need <= 1.05 * least + (vocab + 127) // 128 * 8 * rows
    assert plan(4096, 200256, 4096, F32, True, True, True, True, True)[3] == 9328072960


def test_a_wait_runs_out_by_the_time_that_it_was_looked_at(plan):
    """Four seconds of a wait that is looked at all the time, however the looks lie; a clock
    that went on while nothing ran (for minutes, in the midst of a wait) counts for a
    quarter of a second."""
    ms, start = 10**6, 1 << 60
    for step in (ms // 100, ms, 100 * ms):
        looks = [start + i * step for i in range(4000 * ms // step + 2)]
        assert plan.patience(looks) == len(looks) - 1
    for away in (1000 * ms, 4001 * ms, 600000 * ms, 1 << 62):
        looks, now = [start], start
        for i in range(8):                                 # eight times switched out, or put to sleep
            now += away
            looks.append(now)
            looks += [now + j * ms for j in range(1, 100)]
            now = looks[-1]
        assert plan.patience(looks) == len(looks)
    # nor does a wait whose looks lie far apart go on for ever
    assert plan.patience([start + i * 1000 * ms for i in range(100)]) == 17
