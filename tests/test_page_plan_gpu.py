"""fa_page_plan against the reference plan: every output equal, in place and
replayed, and the refusals that the device makes."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from exact_attention_94_gb300 import ops
from oracle import serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def make(rng, B, ctx_hi, new, P, spare=5):
    """Lengths, a shuffled pool, tables that hold the context's pages."""
    ctx = rng.integers(0, ctx_hi + 1, B)
    new = np.asarray(new if not np.isscalar(new) else rng.integers(0, new + 1, B))
    held, need = -(-ctx // P), -(-(ctx + new) // P)
    blocks = int(max(1, need.max()))
    pages = int(need.sum()) + spare
    order = rng.permutation(pages)
    table = rng.integers(-5, 10 ** 6, (B, blocks))  # entries not yet in use hold anything
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = rng.integers(-9, 10 ** 6, pages)
    free[:pages - at] = order[at:]
    return ctx, new, free, pages - at, table


def check(got, want, table):
    seq, cu, page, slot, pos, left, table_want = want
    for g, w in zip(got, (seq, cu, page, slot, pos, [left])):
        assert g.cpu().tolist() == list(w)
    assert np.array_equal(table.cpu().numpy(), table_want)


@pytest.mark.parametrize("B,ctx_hi,new,P,pad", [
    (1, 0, [1], 16, 0), (1, 0, [0], 16, 0), (1, 0, [0], 16, 3), (1, 33, [500], 16, 1), (7, 100, 40, 16, 9),
    (32, 50, [1] * 32, 4, 0), (33, 64, 3, 1, 31), (1000, 70, 2, 16, 100), (1025, 40, 3, 7, 0), (2500, 9, 5, 32, 5),
    (16384, 6, 1, 4, 11), (3, 1000, [4097, 0, 5000], 64, 700)])
def test_equals_the_reference(B, ctx_hi, new, P, pad):
    rng = np.random.default_rng(B + P)
    ctx, new, free, count, table = make(rng, B, ctx_hi, new, P)
    cap = int(new.sum()) + pad
    want = serving.page_plan(ctx.tolist(), new.tolist(), free.tolist(), count, table, P, cap)
    t = i32(table)
    got = ops.page_plan(i32(ctx), i32(new), i32(free), i32([count]), t, P, cap)
    check(got, want, t)
    assert ops.device_error() == 0


def test_in_place_and_replayed_from_a_graph():
    """The lengths and the free count advance in place; replays take step after step."""
    rng = np.random.default_rng(11)
    B, P, cap, blocks, pages = 40, 16, 8192, 64, 40 * 64
    free = i32(rng.permutation(pages))
    count, lens, new, table = i32([pages]), i32([0] * B), i32([0] * B), i32(np.zeros((B, blocks)))
    out = ops.page_plan(lens, new, free, count, table, P, cap)
    out = out._replace(seq_lens=lens, free_count=count)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.page_plan(lens, new, free, count, table, P, cap, out=out)
    w_lens, w_count, w_table = [0] * B, pages, np.zeros((B, blocks), np.int64)
    for step in range(5):
        n = rng.integers(0, 200, B).tolist() if step % 2 == 0 else [1] * B
        new.copy_(i32(n))
        g.replay()
        want = serving.page_plan(w_lens, n, free.cpu().tolist(), w_count, w_table, P, cap)
        check(out, want, table)
        w_lens, w_count, w_table = want[0], want[5], want[6]
    assert ops.device_error() == 0


@pytest.mark.parametrize("what,code", [("negative", 0x2001), ("context", 0x2001), ("blocks", 0x2001), ("rows", 0x2001),
                                       ("count", 0x2001), ("overflow", 0x2001), ("pages", 0x2002)])
@pytest.mark.parametrize("cap", [300, 9000])
def test_a_step_that_cannot_be_planned_changes_nothing(what, code, cap):
    B, P, pages, blocks = 3, 16, 40, 1000
    ctx, new, count = [5, 0, 17], [20, 7, 100], 30
    if what == "negative":
        new[1] = -1
    if what == "context":
        ctx[0] = -3
    if what == "blocks":
        new[2] = blocks * P
    if what == "rows":
        new[2] = cap
        pages = count = 4000
    if what == "count":
        count = pages + 1
    if what == "overflow":
        ctx[1], new[1] = 2 ** 31 - 1, 2 ** 31 - 1
    if what == "pages":
        count = 7  # eight pages are needed
    table = np.arange(B * blocks).reshape(B, blocks) % 7
    with pytest.raises(serving.PlanError) as e:
        serving.page_plan(ctx, new, [0] * pages, count, table, P, cap)
    assert e.value.code == code
    t = i32(table)
    got = ops.page_plan(i32(ctx), i32(new), i32(range(pages)), i32([count]), t, P, cap)
    assert ops.device_error() == code
    assert got.seq_lens.tolist() == ctx and got.cu_new.tolist() == [0] * 4 and got.free_count.tolist() == [count]
    assert set(got.page.tolist()) == {-1} and set(got.slot.tolist()) == {-1} and set(got.position.tolist()) == {0}
    assert np.array_equal(t.cpu().numpy(), table)


def test_bad_page_numbers_are_reported_and_never_passed_on():
    P = 16
    table = i32([[7, -1, -1], [99, -1, -1]])          # request 1 continues a page that does not exist
    got = ops.page_plan(i32([4, 4]), i32([20, 3]), i32([0, 55, 1, 2, 3, 4, 5, 6]), i32([2]), table, P, 23)
    assert ops.device_error() == 0x2000
    assert got.page.tolist() == [7] * 12 + [-1] * 8 + [-1] * 3   # the stack's top, 55, is no page either
    assert got.slot.tolist() == list(range(4, 16)) + [-1] * 11
    assert table.tolist() == [[7, -1, -1], [99, -1, -1]]


def test_on_another_stream():
    rng = np.random.default_rng(5)
    ctx, new, free, count, table = make(rng, 50, 100, 30, 16)
    cap = int(new.sum())
    want = serving.page_plan(ctx.tolist(), new.tolist(), free.tolist(), count, table, 16, cap)
    s = torch.cuda.Stream()
    args = [i32(x) for x in (ctx, new, free, [count], table)]
    torch.cuda.synchronize()
    got = ops.page_plan(*args, 16, cap, stream=s)
    s.synchronize()
    check(got, want, args[4])


FRESH = """
import sys
import torch
from exact_attention_94_gb300 import ops
i32 = dict(dtype=torch.int32, device="cuda")
for B in map(int, sys.argv[1:]):
    p = ops.page_plan(torch.zeros(B, **i32), torch.ones(B, **i32), torch.arange(B, **i32), torch.full((1,), B, **i32),
                      torch.zeros((B, 1), **i32), 16, B)
    assert p.page.tolist() == list(range(B - 1, -1, -1)) and p.free_count.item() == 0, B
assert ops.device_error() == 0
"""


def test_every_batch_size_launches_in_a_fresh_process():
    """The batches around 48 KiB of shared memory, in rising order: no larger one has gone before."""
    sizes = [1025, 4050, 4051, 4052, 4060, 4094, 4095, 4096, 4097, 16384]
    r = subprocess.run([sys.executable, "-c", FRESH, *map(str, sizes)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_threads_with_batches_of_different_sizes():
    """One thread's batch of 5000 does not take the shared memory from another's of 16384."""
    def plan(B, n, failures):
        with torch.cuda.stream(torch.cuda.Stream()):
            a = [i32([0] * B), i32([1] * B), i32(range(B)), i32([B]), i32([[0]] * B)]
            out = ops.page_plan(*a, 16, B)
            for _ in range(n):
                try:
                    ops.page_plan(*a, 16, B, out=out)
                except Exception as e:  # noqa: BLE001 - the thread's failures are the test's result
                    failures.append(str(e))
            torch.cuda.current_stream().synchronize()
            assert out.page.tolist() == list(range(B - 1, -1, -1))

    failures = []
    threads = [threading.Thread(target=plan, args=(B, 3000, failures)) for B in (4500, 5000, 16384)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, (len(failures), failures[0])
    assert ops.device_error() == 0


def test_finished_requests_give_their_pages_back():
    """Requests come and go in their rows of the table, without the host reading a length: a finished one's pages
    are written behind the stack's top."""
    B, P, pages, blocks, cap = 5, 8, 48, 9, 64
    rng = np.random.default_rng(21)
    free, count, lens, table = i32(rng.permutation(pages)), i32([pages]), i32([0] * B), i32(np.zeros((B, blocks)))
    cols = torch.arange(blocks, device="cuda")
    w_free, w_lens, w_table = free.tolist(), [0] * B, np.zeros((B, blocks), np.int64)
    w_count = pages
    for step in range(30):
        n = rng.integers(0, 12, B).tolist()
        for b in range(B):  # a row whose next tokens do not fit ends, and starts anew
            if w_lens[b] + n[b] > blocks * P or rng.random() < 0.1:
                held = (lens[b] + P - 1) // P
                at = torch.where(cols < held, count + cols, pages + cols)
                spare = torch.cat([free, torch.zeros(blocks, dtype=torch.int32, device="cuda")])
                spare[torch.where(at < pages, at, pages + cols).long()] = table[b]
                free.copy_(spare[:pages])
                count += held
                lens[b] = 0
                w = -(-w_lens[b] // P)
                w_free[w_count:w_count + w] = w_table[b, :w].tolist()
                w_count += w
                w_lens[b] = 0
        p = ops.page_plan(lens, i32(n), free, count, table, P, cap)
        want = serving.page_plan(w_lens, n, w_free, w_count, w_table, P, cap)
        check(p, want, table)
        lens, count = p.seq_lens.clone(), p.free_count.clone()
        w_lens, w_count, w_table = list(want[0]), want[5], want[6]
        live = [int(x) for b in range(B) for x in w_table[b, :-(-w_lens[b] // P)]]
        assert sorted(live + w_free[:w_count]) == list(range(pages))  # every page is held once or free
    assert ops.device_error() == 0


@pytest.mark.parametrize("B", [4095, 16384])
def test_a_large_batch_captured_and_in_place(B):
    lens, count, table = i32([0] * B), i32([2 * B]), i32(np.zeros((B, 2)))
    new, free = i32([1] * B), i32(range(2 * B))
    out = ops.page_plan(lens, new, free, count, table, 1, B)._replace(seq_lens=lens, free_count=count)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.page_plan(lens, new, free, count, table, 1, B, out=out)
    for step in range(2):
        g.replay()
        assert out.page.tolist() == list(range(2 * B - 1 - step * B, B - 1 - step * B, -1))
        assert lens.tolist() == [step + 1] * B and count.item() == (1 - step) * B
    g.replay()                                        # a third token, and no block for it
    assert ops.device_error() == 0x2001 and lens.tolist() == [2] * B and set(out.page.tolist()) == {-1}
