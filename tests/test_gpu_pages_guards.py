"""Page tables: sequences that fall back into pages they have borrowed, pages that cannot be, tokens past
the end.  (The steps in general: test_gpu_serving.py.)"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from test_gpu_kv8 import gen, ints, kv8  # noqa: E402, F401

pytestmark = pytest.mark.gpu

PAGE = 64


def lender_and_borrower(kv8, own, borrowed=4, n_pages=40):
    """Sequence 0 has 300 positions; sequence 1 begins with its first pages and has `own` positions after them."""
    pages = kv8.KV8Pages.all_free(n_pages, PAGE, 2, 12)
    pages = kv8.KV8Pages(pages.table, pages.free, PAGE, pages.lens, pages.held, pages.n_free, ints([0, borrowed]))
    pages.step(ints([300, 0]), 300)
    pages.table[1, :borrowed] = pages.table[0, :borrowed]
    pages.lens[1], pages.held[1] = borrowed * PAGE, borrowed
    pages.step(ints([0, own]), own)
    assert pages.get_error() == 0
    return pages


def whole(pages):
    """Every page of the pool is on the free list or in one sequence's own part of its row, once."""
    n, own = pages.n_free.item(), pages.free[:pages.n_free.item()].tolist()
    for row, held, skip in zip(pages.table.tolist(), pages.held.tolist(), pages.borrowed.tolist()):
        own += row[skip:held]
    return sorted(own) == list(range(pages.free.numel())) and 0 <= n


@pytest.mark.parametrize("keep", [0, 100, 128, 255])
@pytest.mark.parametrize("own", [1, 150])
@pytest.mark.parametrize("new", [1, 200])
def test_no_token_goes_to_a_borrowed_page(kv8, own, keep, new):
    """A sequence that falls back into its prefix, or whose row is used again at once, and adds tokens: recorded,
    and done.  The prefix stays as it was, and all pages of its own come back."""
    from bit_expert_layer_gb300 import _abi
    pages = lender_and_borrower(kv8, own)
    cache = kv8.KV8Cache.empty(40, 2, PAGE, 64, "int8")
    g = gen(keep + own)
    cache.k.copy_(torch.randint(0, 256, cache.k.shape, generator=g, device="cuda", dtype=torch.uint8))
    lent = pages.table[0, :5].long()
    before = [x[lent].clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    t = new + 1
    offsets, positions, slots = pages.step(ints([1, new]), t, keep=ints([256, keep]))
    assert pages.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    assert offsets.tolist() == [0, 1, t] and positions.tolist() == [256] + list(range(keep, keep + new))
    assert slots[1:].tolist() == [-1] * new and slots[0].item() == pages.table[0, 4].item() * PAGE
    assert pages.lens.tolist() == [257, 0] and pages.held.tolist() == [5, 0] and whole(pages)
    # what follows writes none of its tokens, and gives them zeros
    batch = kv8.KV8Batch(pages.table, pages.lens, offsets, new)
    q = torch.randn(t, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
    cache.append(batch, q[:, :2], q[:, 2:])
    for x, was in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        assert torch.equal(x[lent[:4]], was[:4])
    assert torch.isfinite(cache.attention(batch, q)[0]).all() and (cache.attention(batch, q)[1:] == 0).all()
    # the row is free for another request
    pages.borrowed[1] = 0
    pages.step(ints([0, 70]), 70)
    assert pages.get_error() == 0 and pages.lens.tolist() == [257, 70] and whole(pages)


def test_falling_back_and_going_on(kv8):
    """To the end of the borrowed pages and on; into them by whole pages, lowering `borrowed`; done, then another
    request in the row: as the description has it, nothing recorded and no page lost."""
    pages = lender_and_borrower(kv8, 150)
    pages.step(ints([0, 90]), 90, keep=ints([300, 256]))
    assert pages.get_error() == 0 and pages.lens.tolist() == [300, 346] and whole(pages)
    pages.step(ints([0, 0]), 0, keep=ints([300, 128]))
    pages.borrowed[1] = 2
    offsets, positions, slots = pages.step(ints([0, 100]), 100)
    assert pages.get_error() == 0 and pages.held.tolist() == [5, 4] and whole(pages)
    assert not set((slots // PAGE).tolist()) & set(pages.table[0, :5].tolist())
    pages.step(ints([0, 0]), 0, keep=ints([300, 0]))
    pages.borrowed[1] = 0
    pages.step(ints([0, 300]), 300)
    assert pages.get_error() == 0 and pages.held.tolist() == [5, 5] and whole(pages)
    pages.step(ints([0, 0]), 0, keep=ints([0, 0]))
    assert pages.get_error() == 0 and pages.n_free.item() == 40


@pytest.mark.parametrize("count", [13, 2 ** 31 - 1, -1, -2 ** 31])
def test_a_count_of_borrowed_pages_that_cannot_be(kv8, count):
    from bit_expert_layer_gb300 import _abi
    pages = lender_and_borrower(kv8, 20)
    pages.borrowed[1] = count
    pages.step(ints([1, 1]), 2)
    assert pages.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    assert pages.lens.tolist() == [301, 0 if count > 0 else 277]


@pytest.mark.parametrize("bad", [-1, -7, 6, 2 ** 31 - 1])
def test_pages_that_cannot_be_do_not_change_hands(kv8, bad):
    """A held entry out of range that is given back, to the list or straight to another sequence, and an entry of
    the list that is taken: recorded, and -1 from then on."""
    from bit_expert_layer_gb300 import _abi

    def pool(held, table, free, n_free):
        z = [n * PAGE for n in held]
        return kv8.KV8Pages(ints(table), ints(free), PAGE, ints(z), ints(held), ints([n_free]))

    p = pool([2, 1], [[4, bad, 0], [5, 0, 0]], [0, 1, 9, 9, 9, 9], 2)     # to the list
    p.step(ints([0, 0]), 0, keep=ints([0, 64]))
    assert p.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    assert p.n_free.item() == 4 and p.free[:4].tolist() == [0, 1, 4, -1]
    assert p.step(ints([1, 0]), 1, keep=ints([0, 64]))[2].tolist() == [-1]     # what the list has is taken
    assert p.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS and p.table[0, 0].item() == -1
    p = pool([2, 1], [[4, bad, 0], [5, 0, 0]], [0, 1, 9, 9, 9, 9], 2)     # from hand to hand
    slots = p.step(ints([0, 70]), 70, keep=ints([0, 64]))[2].tolist()
    assert p.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    assert p.table[1].tolist() == [5, -1, 4] and slots == [-1] * 64 + [4 * PAGE + i for i in range(6)]
    p = pool([0, 1], [[0, 0, 0], [5, 0, 0]], [0, bad, 9, 9, 9, 9], 2)     # from the list
    assert p.step(ints([1, 0]), 1)[2].tolist() == [-1] and p.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    assert p.table[0, 0].item() == -1 and p.n_free.item() == 1


def test_control_is_checked(kv8):
    """Like the other tensors, before anything is launched."""
    p = kv8.KV8Pages.all_free(6, PAGE, 2, 3)
    zeros = lambda *s, **kw: torch.zeros(*s, **dict(dict(dtype=torch.int32, device="cuda"), **kw))  # noqa: E731
    for control in (zeros(2, device="cpu"), zeros(1), zeros(0), zeros(2, dtype=torch.int64), zeros(2, dtype=torch.float32),
                    zeros(1, 2), zeros(4)[::2]):
        with pytest.raises(ValueError):
            kv8.KV8Pages(p.table, p.free, PAGE, p.lens, p.held, p.n_free, control=control)
    for control in (zeros(2), zeros(5), zeros(2, dtype=torch.uint32)):
        q = kv8.KV8Pages(p.table, p.free, PAGE, p.lens, p.held, p.n_free, control=control)
        q.fork()
        assert q.control is control and q.step(ints([0, 0]), 0)[0].tolist() == [0, 0, 0] and q.get_error() == 0


def test_tokens_past_the_rows_and_past_the_table(kv8):
    """Recorded; the others keep their rows and positions, nothing that is cached moves, and what follows leaves out
    the tokens past the table and the sequences whose rows do not exist."""
    from bit_expert_layer_gb300 import _abi
    pages = kv8.KV8Pages.all_free(20, PAGE, 3, 4)
    cache = kv8.KV8Cache.empty(20, 1, PAGE, 64, "int8")
    g = gen(5)
    rows = lambda n: torch.randint(-127, 128, (n, 2, 64), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731

    def append(new, n_tokens, max_new):
        offsets, positions, slots = pages.step(ints(new), n_tokens)
        x = rows(n_tokens)
        cache.append(kv8.KV8Batch(pages.table, pages.lens, offsets, max_new), x[:, :1], x[:, 1:])
        return offsets.tolist(), positions.tolist(), slots, x

    append([250, 10, 20], 280, 250)
    codes = cache.k.clone()
    *_, slots, x = append([10, 3, 4], 17, 10)             # the first one ends at 260 of 256
    assert pages.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS and cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    assert pages.lens.tolist() == [260, 13, 24] and pages.held.tolist() == [4, 1, 1]
    assert slots[6:10].tolist() == [-1] * 4 and (slots[:6] >= 0).all() and (slots[10:] >= 0).all()
    at = torch.cat([slots[:6], slots[10:]]).long()
    changed = (cache.k != codes).any(-1).squeeze(1).flatten().nonzero().flatten().tolist()
    blocks = {i // 16 for i in at.tolist()}               # (older codes of a block change with its scale)
    assert {i // 16 for i in changed} <= blocks
    scale = cache.k_scale.view(-1)[at // 16]
    values = cache.k.view(torch.int8).view(-1, 64)[at].float() * scale[:, None]
    assert torch.equal(values, torch.cat([x[:6, 0], x[10:, 0]]).float())
    codes = cache.k.clone()
    offsets, positions, slots, x = append([0, 5, 6], 7, 6)     # 11 tokens, 7 rows: the last sequence's do not fit
    assert pages.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS and cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    assert offsets == [0, 0, 5, 11] and positions == [13, 14, 15, 16, 17, 24, 25]
    assert pages.lens.tolist() == [256, 18, 30]
    changed = (cache.k != codes).any(-1).squeeze(1).flatten().nonzero().flatten()
    assert set((changed // PAGE).tolist()) == {pages.table[1, 0].item()}
