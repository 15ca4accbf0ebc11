"""Page tables (afx_kv_tables) against a list-and-stack simulation, and cache
writes (afx_kv_write) against indexing.  Whole numbers and copies: equal."""
import random

import pytest

import serving_ref as ref

pytestmark = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _state(n, page, old, new, seed, spare=3, cols_extra=1):
    rng = random.Random(seed)
    cols = max(1, max(ref.pages(max(o, w), page) for o, w in zip(old, new))) + cols_extra
    held = sum(ref.pages(o, page) for o in old)
    need = sum(max(0, ref.pages(w, page) - ref.pages(o, page)) for o, w in zip(old, new))
    ids = list(range(held + need + spare))
    rng.shuffle(ids)
    table, at = [], 0
    for o in old:
        k = ref.pages(o, page)
        table.append(ids[at:at + k] + [-7] * (cols - k))
        at += k
    stack = ids[at:] + [-9] * held
    return table, stack, len(ids) - held


def _call(afx, page, old, new, table, stack, count, max_tokens, status=None):
    import torch
    d = {"table": _ints(table), "stack": _ints(stack), "count": _ints([count]), "out": _ints([-5]),
         "starts": _ints([-5] * (len(old) + 1)), "slots": _ints([-5] * max_tokens), "positions": _ints([-5] * max_tokens)}
    afx.afx_kv_tables(page, _ints(old), _ints(new), d["table"], d["stack"], d["count"], d["out"], d["starts"], d["slots"],
                      d["positions"], status_dev=status)
    torch.cuda.synchronize()
    return {k: v.tolist() for k, v in d.items()}


def _check(got, want):
    table, stack, count, starts, slots, positions = want
    assert got["out"] == [count]
    assert got["starts"] == starts
    assert got["slots"] == slots
    assert got["positions"] == positions
    assert got["table"] == table
    assert got["stack"] == stack


def _lengths(n, page, kind, rng):
    old = [rng.choice([0, 0, 1, page - 1, page, page + 1, rng.randint(0, 5 * page)]) for _ in range(n)]
    if kind == "step":
        new = [o + 1 for o in old]
    elif kind == "still":
        new = list(old)
    elif kind == "end":
        new = [0] * n
    elif kind == "start":
        old, new = [0] * n, [rng.randint(0, 4 * page) for _ in range(n)]
    else:
        new = [rng.choice([0, o, o + 1, max(0, o - 3), o + rng.randint(0, 6 * page)]) for o in old]
    return old, new


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", ["step", "still", "end", "start", "mixed"])
@pytest.mark.parametrize("n", [1, 7, 1025])
def test_tables_match_the_simulation(afx, n, kind, page):
    import torch
    rng = random.Random(n * 1000 + page)
    old, new = _lengths(n, page, kind, rng)
    table, stack, count = _state(n, page, old, new, seed=page + n)
    tokens = sum(max(0, w - o) for o, w in zip(old, new)) + rng.choice([0, 1, 37])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _call(afx, page, old, new, table, stack, count, tokens, status)
    assert status.item() == 0
    _check(got, ref.kv_tables(page, old, new, table, stack, count, tokens))


def test_tables_of_the_most_requests(afx):
    rng = random.Random(5)
    n = afx.AFX_KV_MAX_REQUESTS
    old = [rng.randint(0, 90) for _ in range(n)]
    new = [rng.choice([0, o + 1, max(0, o - 20), o + 40]) for o in old]
    table, stack, count = _state(n, 16, old, new, seed=3)
    tokens = sum(max(0, w - o) for o, w in zip(old, new))
    _check(_call(afx, 16, old, new, table, stack, count, tokens), ref.kv_tables(16, old, new, table, stack, count, tokens))


def test_pages_given_back_serve_the_same_call(afx):
    """No page is free at the start: growth takes what shrinking requests return, last first."""
    old, new = [64, 0, 48, 5], [0, 40, 10, 33]
    table, stack, count = _state(4, 16, old, new, seed=1, spare=0)
    stack, count = [-9] * len(stack), 0
    tokens = 40 + 28
    got = _call(afx, 16, old, new, table, stack, count, tokens)
    _check(got, ref.kv_tables(16, old, new, table, stack, count, tokens))
    assert got["out"] == [6 - 5]


def test_steps_follow_one_another(afx):
    """Many steps on one pool: no page is lost or handed out twice."""
    rng = random.Random(9)
    n, page, cols, total = 12, 16, 20, 150
    table, stack, count, lens = [[-1] * cols for _ in range(n)], list(range(total)), total, [0] * n
    for _ in range(40):
        new = [rng.choice([x + 1, x + 1, x + 9, 0, max(0, x - 4)]) if x < 280 else 0 for x in lens]
        need = sum(ref.pages(w, page) for w in new)
        if need > total:
            new = [min(w, x) for w, x in zip(new, lens)]
        tokens = sum(max(0, w - x) for x, w in zip(lens, new)) + 2
        got = _call(afx, page, lens, new, table, stack, count, tokens)
        _check(got, ref.kv_tables(page, lens, new, table, stack, count, tokens))
        table, stack, count, lens = got["table"], got["stack"], got["out"][0], new
        held = [p for r in range(n) for p in table[r][:ref.pages(lens[r], page)]]
        assert sorted(held + stack[:count]) == list(range(total))


@pytest.mark.parametrize("what", ["pages", "negative old", "negative new", "past the row", "tokens", "count high",
                                  "count negative", "given back twice"])
def test_a_call_that_cannot_be_served_changes_nothing(afx, what):
    import torch
    old, new = [20, 0, 33], [21, 50, 0]
    table, stack, count = _state(3, 16, old, new, seed=2, spare=0)
    tokens, bit = 51, afx.AFX_DEV_BAD_LENGTH
    if what == "pages":
        new, tokens, bit = [21, 112, 33], 113, afx.AFX_DEV_NO_PAGES
        table = [r + [-7] * (8 - len(r)) for r in table]
    elif what == "negative old":
        old = [20, -1, 33]
    elif what == "negative new":
        new = [21, -50, 0]
    elif what == "past the row":
        new = [21, 16 * len(table[0]) + 1, 0]
        tokens = 500
    elif what == "tokens":
        tokens = 50
    elif what == "count high":
        count = len(stack) + 1
    elif what == "count negative":
        count = -1
    else:
        new, count = [0, 0, 0], len(stack)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _call(afx, 16, old, new, table, stack, count, tokens, status)
    assert status.item() == bit
    assert got["table"] == table and got["stack"] == stack and got["out"] == [count]
    assert got["starts"] == [0] * 4 and got["slots"] == [-1] * tokens and got["positions"] == [-1] * tokens


def test_a_page_outside_the_pool_gives_no_slot(afx):
    import torch
    old, new = [20, 16], [22, 18]
    table = [[1, 1000, -7], [2, -7, -7]]
    stack, count = [0, 3, -4, -9], 3  # the top of the stack is no page
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _call(afx, 16, old, new, table, stack, count, 4, status)
    assert status.item() == afx.AFX_DEV_BAD_PAGE
    assert got["slots"] == [-1] * 4 and got["positions"] == [20, 21, 16, 17]


def test_tables_refuse_bad_arguments(afx):
    good = [_ints([1]), _ints([2]), _ints([[0, 0]]), _ints([0, 1]), _ints([2]), _ints([0]), _ints([0, 0]), _ints([0]), _ints([0])]

    def call(**change):
        a = list(good)
        for i, v in change.items():
            a[int(i[1:])] = v
        afx.afx_kv_tables(16, *a)

    call()
    for change in ({"a5": good[4]},):  # the count in and out at one place
        with pytest.raises(afx.AfxError) as err:
            call(**change)
        assert err.value.status == afx.AFX_E_ARG
    for change in ({"a0": good[0].long()}, {"a6": _ints([0])}, {"a2": _ints([0, 0])}, {"a7": _ints([0, 0])}, {"a1": good[1].cpu()}):
        with pytest.raises(ValueError):
            call(**change)
    with pytest.raises(afx.AfxError):
        afx.afx_kv_tables(17, *good)


# ---- cache writes ----------------------------------------------------------------

_LAYOUTS = {"tokens, heads": (0, 1, 2, 3), "heads, tokens": (0, 2, 1, 3), "head pools": (2, 0, 1, 3)}


def _pools(pages, page, heads, dim, dtype, layout, seed):
    """Two pools of logical shape [page][token][head][dim] stored in another order."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    order = _LAYOUTS[layout]
    shape = (pages, page, heads, dim)
    made = [torch.randn([shape[i] for i in order], generator=g, device="cuda").to(dtype) for _ in range(2)]
    return [m.permute([order.index(i) for i in range(4)]) for m in made]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("layout", list(_LAYOUTS))
@pytest.mark.parametrize("tokens,heads,page,shift", [(1, 1, 16, 0), (33, 8, 16, 0), (300, 2, 128, 1), (77, 5, 64, 8)])
def test_writes_land_in_their_slots(afx, dtype, dim, layout, tokens, heads, page, shift):
    import torch
    dtype = getattr(torch, dtype)
    pages = ref.pages(tokens, page) + 2
    k_pool, v_pool = _pools(pages, page, heads, dim, dtype, layout, seed=tokens)
    rows = torch.randn((tokens, 2 * heads * dim + 3 * shift + 8), device="cuda").to(dtype)
    k = rows[:, shift:shift + heads * dim].unflatten(1, (heads, dim))  # an odd shift: rows off any alignment
    v = rows[:, shift + heads * dim:shift + 2 * heads * dim].unflatten(1, (heads, dim))
    slots = torch.randperm(pages * page, device="cuda")[:tokens].to(torch.int32)
    slots[tokens // 2] = -1
    want = [p.clone() for p in (k_pool, v_pool)]
    for w, x in zip(want, (k, v)):
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                w[s // page, s % page] = x[t]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    afx.afx_kv_write(afx.kv_cache(k_pool, v_pool), k, v, slots, status_dev=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert torch.equal(k_pool, want[0]) and torch.equal(v_pool, want[1])


def test_a_slot_past_the_pool_is_flagged_and_skipped(afx):
    import torch
    k_pool, v_pool = _pools(3, 16, 2, 64, torch.bfloat16, "tokens, heads", 1)
    x = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    want = k_pool.clone()
    want[0, 5] = x[2]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    afx.afx_kv_write(afx.kv_cache(k_pool, v_pool), x, x, _ints([48, 2**31 - 1, 5]), status_dev=status)
    torch.cuda.synchronize()
    assert status.item() == afx.AFX_DEV_BAD_PAGE
    assert torch.equal(k_pool, want)


def test_a_write_of_no_tokens_is_no_work(afx):
    import torch
    k_pool, v_pool = _pools(1, 16, 1, 64, torch.float16, "tokens, heads", 1)
    x = torch.empty((0, 1, 64), dtype=torch.float16, device="cuda")
    afx.afx_kv_write(afx.kv_cache(k_pool, v_pool), x, x, _ints([]))


def test_writes_past_4_gib(afx):
    import torch
    pages, page, heads, dim = 20_000, 128, 8, 128  # 5.2 GB a pool
    k_pool, v_pool = [torch.zeros((pages, page, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x = torch.randn((2, heads, dim), device="cuda").to(torch.bfloat16)
    afx.afx_kv_write(afx.kv_cache(k_pool, v_pool), x, x, _ints([pages * page - 1, 3]))
    torch.cuda.synchronize()
    assert torch.equal(k_pool[-1, -1], x[0]) and torch.equal(v_pool[0, 3], x[1])
    assert k_pool.count_nonzero() == 2 * heads * dim


def test_writes_refuse_bad_arguments(afx):
    import torch
    k_pool, v_pool = _pools(3, 16, 2, 64, torch.bfloat16, "tokens, heads", 1)
    x = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    cache = afx.kv_cache(k_pool, v_pool)
    for bad in ((cache, x.half(), x.half(), _ints([0, 1, 2])), (cache, x, x[:2], _ints([0, 1, 2])),
                (cache, x[:, :1], x[:, :1], _ints([0, 1, 2])), (cache, x, x, _ints([0, 1])), (cache, x.cpu(), x, _ints([0, 1, 2]))):
        with pytest.raises(ValueError):
            afx.afx_kv_write(*bad)
    for pools in ((k_pool.float(), v_pool.float()), (k_pool, v_pool[:2]), (k_pool[0], v_pool[0]),
                  (k_pool.permute(0, 1, 3, 2), v_pool.permute(0, 1, 3, 2))):
        with pytest.raises(ValueError):
            afx.kv_cache(*pools)
    for pools in ([p[:, :12] for p in (k_pool, v_pool)], [p[..., :32] for p in (k_pool, v_pool)]):
        with pytest.raises(afx.AfxError) as err:
            afx.afx_kv_write(afx.kv_cache(*pools), *[torch.zeros((3, 2, pools[0].shape[3]), dtype=torch.bfloat16, device="cuda")] * 2,
                             _ints([0, 1, 2]))
        assert err.value.status == afx.AFX_E_ARG
