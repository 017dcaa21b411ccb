"""GPU: pages and slots of a step against one request after another in Python integers."""
import numpy as np
import pytest
import torch

import _step_ref as ref
import block_scaled_fp8_weight_gb300 as bsf8

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def books(r, B, table_pages, pool, held):
    """Books in which requests hold pages and the stack the others, in any order; stale entries everywhere."""
    order = r.permutation(pool)
    table = r.integers(-5, 5, size=(B, table_pages)).astype(np.int64)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = r.integers(-9, 0, size=pool)
    free[:pool - at] = order[at:]
    return table, np.array(held), free, pool - at


def check(state, lens, add, done, page, tokens, status=0):
    table, held, free, count = state
    book = bsf8.PageBook(i32(table), i32(held), i32(free), i32([count]))
    out = bsf8.kv_plan(book, i32(lens), i32(add), page_size=page, tokens=tokens, done=None if done is None else i32(done))
    want = ref.plan(table, held, free, count, lens, add, done, page, tokens)
    got = dict(zip(("req", "slot", "start", "granted"), out), table=book.table, held=book.held, free=book.free, count=book.count)
    for name, t in got.items():
        assert np.array_equal(t.cpu().numpy().reshape(np.shape(want[name])), want[name]), name
    assert bsf8.device_status() == status
    return want


@pytest.mark.parametrize("B,page,most,longest,tight", [
    (1, 16, 1, 0, 1.0), (1, 64, 1, 9000, 1.0), (7, 16, 9, 0, 1.0), (33, 48, 64, 300, 0.9), (64, 16, 1, 100, 1.0),
    (65, 32, 5, 500, 0.7), (300, 16, 3, 200, 0.97), (1023, 64, 1, 700, 1.0), (1024, 16, 2, 64, 0.5), (1024, 1024, 1, 5000, 1.0)])
@pytest.mark.parametrize("leave", [0.0, 0.4, 1.0])
def test_plan(bsf8_lib, B, page, most, longest, tight, leave):
    r = np.random.default_rng(B + page)
    lens = r.integers(0, 40 * page // 16, size=B)
    held = -(-lens // page) + r.integers(0, 2, size=B)  # some hold a page for drafts that were not kept
    done = (r.random(B) < leave).astype(int)
    add = r.integers(0, most + 1, size=B)
    if longest:
        add[r.integers(0, B)] = longest
    lens = np.where(done, 0, lens)
    table_pages = int(max(held.max(), (-(-(lens + add) // page)).max()))
    want = sum(max(0, -(-(n + a) // page) - (0 if d else h)) for n, a, h, d in zip(lens, add, held, done))
    spare = max(0, int(tight * want) - int(held[done > 0].sum()))
    state = books(r, B, table_pages, int(held.sum()) + spare + 1, held)
    w = check(state, lens, add, done, page, int(add.sum()) + 3)
    assert tight < 1 or w["granted"].sum() == add.sum()
    check(state, lens, add, None if leave == 0 else done, page, int(0.8 * add.sum()))  # a token budget that runs out


def test_nothing_to_do_and_no_tokens(bsf8_lib):
    r = np.random.default_rng(0)
    state = books(r, 5, 4, 20, [0, 1, 4, 2, 0])
    check(state, [0, 16, 64, 20, 0], [0] * 5, None, 16, 0)
    check(state, [0, 16, 64, 20, 0], [0] * 5, [1] * 5, 16, 7)     # all leave
    # no room for a token: none granted (and the third row's 65th would be past its table)
    check(state, [0, 16, 64, 20, 0], [1] * 5, None, 16, 0, 10)


def test_a_request_that_needs_no_page_goes_on_while_others_wait(bsf8_lib):
    r = np.random.default_rng(1)
    w = check(books(r, 4, 8, 6, [1, 2, 1, 1]), [16, 20, 16, 3], [1, 4, 40, 5], None, 16, 99)
    assert list(w["granted"]) == [1, 4, 0, 5] and w["count"] == 0


def test_what_comes_back_is_handed_out_again(bsf8_lib):
    """An empty stack, a row that leaves and the request that takes its place in the same call."""
    r = np.random.default_rng(2)
    w = check(books(r, 3, 6, 9, [4, 0, 5]), [0, 0, 0], [90, 33, 7], [1, 0, 1], 16, 200)
    assert list(w["granted"]) == [90, 33, 0]


def test_bad_books_and_lengths_are_cut_off_and_reported(bsf8_lib):
    INDEX = 10
    r = np.random.default_rng(3)
    state = books(r, 4, 4, 20, [1, 1, 1, 1])
    for lens, add in (([0, -1, 0, 0], [1, 1, 1, 1]), ([0, 0, 0, 0], [1, -1, 1, 1]), ([0, 60, 0, 0], [1, 5, 1, 1]),
                      ([0, 2 ** 31 - 1, 0, 0], [1, 2 ** 31 - 1, 1, 1])):
        check(state, lens, add, [0, 0, 1, 0], 16, 9, INDEX)
    table, held, free, count = state
    for bad in (-3, 5):  # a row that claims more pages than it can hold
        want = held.copy()
        want[1] = max(0, min(bad, 4))
        book = bsf8.PageBook(i32(table), i32([1, bad, 1, 1]), i32(free), i32([count]))
        bsf8.kv_plan(book, i32([0] * 4), i32([0] * 4), page_size=16, tokens=1)
        assert book.held.tolist() == list(want) and bsf8.device_status() == INDEX
    for bad in (-1, 21):
        book = bsf8.PageBook(i32(table), i32(held), i32(free), i32([bad]))
        bsf8.kv_plan(book, i32([0] * 4), i32([0] * 4), page_size=16, tokens=1)
        assert book.count.tolist() == [max(0, min(bad, 20))] and bsf8.device_status() == INDEX
    # more pages come back than the stack has room for
    book = bsf8.PageBook(i32(table), i32([4, 4, 4, 4]), i32(free), i32([10]))
    bsf8.kv_plan(book, i32([0] * 4), i32([0] * 4), page_size=16, tokens=1, done=i32([1] * 4))
    assert book.count.tolist() == [20] and book.free.tolist()[10:] == list(table.reshape(-1)[:10])
    assert bsf8.device_status() == INDEX


@pytest.mark.parametrize("B,pages", [(64, 64), (64, 65), (128, 32), (128, 33), (1, 4096), (1, 4097), (3, 8191), (64, 2048), (128, 700)])
@pytest.mark.parametrize("leave", [None, 0.0, 0.3, 1.0])
def test_long_requests_leave_in_a_call_of_few_tokens(bsf8_lib, B, pages, leave):
    """Few new tokens, tables on both sides of where the kernel for many pages takes over."""
    r = np.random.default_rng(B + pages)
    held = np.maximum(1, pages - r.integers(0, 3, size=B))
    done = None if leave is None else (r.random(B) < leave).astype(int)
    lens = held * 16 - r.integers(0, 16, size=B)
    if done is not None:
        lens = np.where(done, 0, lens)
    add = np.minimum(r.integers(0, 9, size=B), pages * 16 - lens)
    w = check(books(r, B, pages, int(held.sum()) + 2 * B, held), lens, add, done, 16, int(add.sum()) + 1)
    assert (w["granted"] == add).all()


@pytest.mark.parametrize("N", [(1 << 30) - 2, (1 << 30) - 1, 1 << 30])
@pytest.mark.parametrize("B,large", [(4, (0, 1)), (7, (0, 1, 2)), (40, (0, 5, 35)), (200, (3, 7, 40, 190)), (200, (0, 1, 2, 3, 4))])
def test_requests_past_the_largest_budget_leave_nothing_behind_them(bsf8_lib, N, B, large):
    """Requests that each ask for more tokens than any call has: what comes after them does not fit either, though it needs no
    page."""
    pages = (1 << 30) // 1024 + 1
    add, held = [0] * B, [0] * B
    for b in large:
        add[b] = N + 1
        if b + 1 not in large:
            add[b + 1], held[b + 1] = 5, 1
    add[B - 1], held[B - 1] = 3, 1
    book = bsf8.PageBook(torch.zeros((B, pages), dtype=torch.int32, device="cuda"), i32(held), i32([2, 1, 0]), i32([3]))
    req, slot, start, granted = bsf8.kv_plan(book, i32([0] * B), i32(add), page_size=1024, tokens=N)
    assert not granted.any() and not start.any() and not req.any() and (slot == -1).all()
    assert int(book.count) == 3 and book.held.tolist() == held and bsf8.device_status() == 0


def test_fresh_books_serve_a_few_steps(bsf8_lib):
    """Steps one after another from PageBook.empty: no page is held twice, none is lost."""
    r = np.random.default_rng(4)
    B, page, pool = 13, 32, 60
    book = bsf8.PageBook.empty(B, 16, pool)
    lens = np.zeros(B, int)
    for step in range(12):
        done = (r.random(B) < 0.2).astype(int)
        lens[done > 0] = 0
        add = np.where(lens == 0, r.integers(1, 200, size=B), r.integers(1, 10, size=B))
        add = np.minimum(add, 16 * page - lens)
        granted = bsf8.kv_plan(book, i32(lens), i32(add), page_size=page, tokens=1500, done=i32(done))[3].cpu().numpy()
        lens = lens + granted
        held, table = book.held.cpu().numpy(), book.table.cpu().numpy()
        assert (held * page >= lens).all()
        have = np.concatenate([table[b, :held[b]] for b in range(B)] + [book.free.cpu().numpy()[:int(book.count)]])
        assert sorted(have.tolist()) == list(range(pool))
    assert bsf8.device_status() == 0


def test_plan_in_a_graph(bsf8_lib):
    """Captured and replayed: each replay goes on from the books as the one before left them."""
    book = bsf8.PageBook.empty(3, 8, 20)
    lens, add = i32([0, 0, 0]), i32([20, 5, 1])
    bsf8.kv_plan(bsf8.PageBook.empty(3, 8, 20), lens, add, page_size=16, tokens=32)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        req, slot, start, granted = bsf8.kv_plan(book, lens, add, page_size=16, tokens=32)
        lens += granted
    table, held, free, count = (t.cpu().numpy().copy() for t in (book.table, book.held, book.free, book.count))
    n = np.zeros(3, int)
    for _ in range(4):
        g.replay()
        w = ref.plan(table, held, free, int(np.ravel(count)[0]), n, [20, 5, 1], None, 16, 32)
        table, held, free, count = w["table"], w["held"], w["free"], np.array([w["count"]])
        assert np.array_equal(req.cpu().numpy(), w["req"]) and np.array_equal(slot.cpu().numpy(), w["slot"])
        assert np.array_equal(book.table.cpu().numpy(), table) and np.array_equal(book.held.cpu().numpy(), held)
        n = n + w["granted"]
        assert np.array_equal(lens.cpu().numpy(), n)
