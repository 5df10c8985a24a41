"""paged_extend and paged_release against a plain model of the block list:
whole numbers, equal in every entry, at the sizes and states where they can go
wrong (nothing new, blocks that run out, tables that are full, padded rows)."""

import pytest
import torch

from exact_softmax_attention_causal_b200 import AttnError, paged_extend, paged_release

pytestmark = pytest.mark.gpu

I32 = torch.int32


def extend_ref(lens, new, table, free, num_free, bs, num_blocks, max_tokens):
    """One sequence, one block, one row at a time."""
    table = [row[:] for row in table]
    F = num_free if 0 <= num_free <= len(free) else 0
    flag = F != num_free
    out, cu, pos, slots, taken, rows, short = [], [], [], [], 0, 0, False
    for b, (L, n) in enumerate(zip(lens, new)):
        cu.append(min(rows, max_tokens))
        ok = L >= 0 and n >= 0 and L + n <= len(table[0]) * bs
        count = max(n, 0)
        need = -(-(L + n) // bs) - -(-L // bs) if ok else 0
        short |= need > 0 and taken + need > F
        if short and need:
            ok = False
        if count and rows + count > max_tokens:
            ok = False
        got = []
        if ok:
            for i in range(need):
                e = free[F - 1 - taken - i]
                if not 0 <= e < num_blocks:
                    e, flag = -1, True
                table[b][-(-L // bs) + i] = e
                got.append(e)
        if L >= 0 and n >= 0 and L + n <= len(table[0]) * bs:
            taken += need  # the running sum goes on, so that nothing behind a shortage is served
        for i in range(count):
            if rows + i >= max_tokens:
                break
            e = table[b][(L + i) // bs] if ok else -1
            if ok and not 0 <= e < num_blocks:
                e, flag = -1, True
            pos.append(L + i if ok else 0)
            slots.append(e * bs + (L + i) % bs if e >= 0 else -1)
        rows += count
        flag |= not ok
        out.append(L + n if ok else (L if L < 0 else -1 - L))
    cu.append(min(rows, max_tokens))
    pos += [0] * (max_tokens - len(pos))
    slots += [-1] * (max_tokens - len(slots))
    served = sum(-(-(L + n) // bs) - -(-L // bs) for L, n, o in zip(lens, new, out) if o >= 0)
    return table, out, num_free - served, cu, pos, slots, flag


def _state(B, bs, max_blocks, num_blocks, seed, hi, new_hi, extra=50):
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, hi + 1, (B,), generator=g)
    new = torch.randint(0, new_hi + 1, (B,), generator=g)
    perm = torch.randperm(num_blocks, generator=g).tolist()
    table = [[-7] * max_blocks for _ in range(B)]
    at = 0
    for b in range(B):
        for j in range(-(-int(lens[b]) // bs)):
            table[b][j] = perm[at]
            at += 1
    free = perm[at:] + [-9] * extra
    return lens.tolist(), new.tolist(), table, free, len(perm) - at


def _t(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def _check_extend(lens, new, table, free, num_free, bs, num_blocks, max_tokens, in_place=False, stream=None):
    ref = extend_ref(lens, new, table, free, num_free, bs, num_blocks, max_tokens)
    L, n, tb, fr, nf = _t(lens), _t(new), _t(table), _t(free), _t([num_free])
    status = torch.zeros(1, dtype=I32, device="cuda")
    kw = dict(seq_lens_out=L, num_free_out=nf) if in_place else {}
    torch.cuda.synchronize()
    lo, nfo, cu, pos, slots = paged_extend(L, n, tb, fr, nf, bs, num_blocks, max_tokens, status=status,
                                           stream=stream, **kw)
    torch.cuda.synchronize()
    assert tb.tolist() == ref[0]
    assert lo.tolist() == ref[1]
    assert nfo.tolist() == [ref[2]]
    assert cu.tolist() == ref[3]
    assert pos.tolist() == ref[4]
    assert slots.tolist() == ref[5]
    assert bool(status.item() & 1) == ref[6]
    assert fr.tolist() == free
    if in_place:
        assert lo.data_ptr() == L.data_ptr() and nfo.data_ptr() == nf.data_ptr()
    else:
        assert L.tolist() == lens and nf.tolist() == [num_free]


@pytest.mark.parametrize("B,bs,hi,new_hi,pad", [(1, 16, 0, 1, 0), (1, 16, 40, 33, 0), (7, 1, 9, 5, 3), (64, 16, 700, 1, 5),
                                                (300, 48, 900, 200, 1000), (1025, 128, 300, 9, 0), (2500, 7, 20, 0, 11)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(B, bs, hi, new_hi, pad, in_place):
    max_blocks = -(-(hi + new_hi) // bs) + 2
    lens, new, table, free, nf = _state(B, bs, max_blocks, B * max_blocks + 5, B, hi, new_hi)
    _check_extend(lens, new, table, free, nf, bs, B * max_blocks + 5, sum(new) + pad, in_place)


@pytest.mark.parametrize("B", [4010, 4011, 8192])
def test_the_most_sequences(B):
    """Around the batch that fills the shared memory a kernel has unasked, and the largest."""
    lens, new, table, free, nf = _state(B, 16, 4, B * 4, B, 40, 5)
    _check_extend(lens, new, table, free, nf, 16, B * 4, sum(new) + 3, in_place=True)
    lens, _, table, free, nf = _state(B, 16, 4, B * 4, B + 1, 60, 0, extra=B * 4)
    _check_release(lens, [b % 2 for b in range(B)], table, free, nf, 16, B * 4)


def test_extend_fills_every_block_to_its_edge():
    # lengths around a block's end, new tokens around whole blocks
    lens = [0, 15, 16, 17, 31, 32, 0, 16, 47, 48]
    new = [16, 1, 1, 15, 1, 0, 0, 32, 1, 17]
    table = [[-7] * 6 for _ in lens]
    at = 0
    for b, L in enumerate(lens):
        for j in range(-(-L // 16)):
            table[b][j] = at
            at += 1
    free = list(range(at, at + 12))
    _check_extend(lens, new, table, free, 12, 16, at + 12, sum(new))


@pytest.mark.parametrize("num_free", [0, 1, 2, 5, 9, 10, 11, -1, 40])
def test_extend_runs_out_of_blocks(num_free):
    # 10 blocks are asked for, some sequences ask for none
    lens, new = [3, 0, 16, 14, 0, 30, 7], [1, 40, 17, 1, 0, 3, 60]
    table, at = [[-7] * 8 for _ in lens], 0
    for b, L in enumerate(lens):
        for j in range(-(-L // 16)):
            table[b][j] = at
            at += 1
    _check_extend(lens, new, table, list(range(at, at + 15)), num_free, 16, at + 15, 130)


@pytest.mark.parametrize("max_tokens", [0, 1, 9, 10, 11, 29, 30, 31])
def test_extend_with_more_tokens_than_rows(max_tokens):
    lens, new, table, free, nf = [0, 5, 0, 8], [10, 10, 0, 10], [[-7] * 4, [1, -7, -7, -7], [-7] * 4, [0, -7, -7, -7]], \
        [2, 3, 4, 5, 6], 5
    _check_extend(lens, new, table, free, nf, 16, 7, max_tokens)


def test_extend_bad_values_are_marked_and_the_rest_is_served():
    # negative length, negative count, too long for the table, entries outside the pool
    lens = [-3, 4, 60, 20, 5, 2 ** 31 - 1]
    new = [2, -2, 10, 3, 20, 2 ** 31 - 1]
    table = [[0, 1, 2, 3], [4, -7, -7, -7], [5, 6, 7, 8], [9, 99, -7, -7], [10, -7, -7, -7], [-7] * 4]
    _check_extend(lens, new, table, [50, 11], 2, 16, 12, 60)


def test_extend_many_rows_over_the_cluster():
    lens, new, table, free, nf = _state(40, 16, 300, 13000, 5, 1000, 3000)
    _check_extend(lens, new, table, free, nf, 16, 13000, sum(new) + 4000, in_place=True)


def release_ref(lens, fin, table, free, num_free, bs, num_blocks):
    free, F, flag, out = free[:], num_free, False, []
    if not 0 <= F <= len(free):
        F, flag = len(free), True
    given = 0
    for b, L in enumerate(lens):
        out.append(0 if fin[b] else L)
        if not fin[b]:
            continue
        held = -1 - L if L < 0 else L
        if held > len(table[0]) * bs:
            flag = True
            continue
        for j in range(-(-held // bs)):
            if F + given >= len(free):
                flag = True
                break
            free[F + given] = table[b][j]
            flag |= not 0 <= table[b][j] < num_blocks
            given += 1
    return out, free, num_free + given, flag


@pytest.mark.parametrize("B,bs,hi", [(1, 16, 100), (5, 1, 30), (64, 16, 900), (700, 128, 5000), (2100, 16, 40)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release(B, bs, hi, in_place):
    max_blocks = -(-hi // bs) + 1
    lens, _, table, free, nf = _state(B, bs, max_blocks, B * max_blocks, B, hi, 0, extra=B * max_blocks)
    fin = [(b * 7) % 3 == 0 for b in range(B)]
    lens[B // 2] = -1 - lens[B // 2]  # as a failed extension leaves it
    _check_release(lens, [int(f) * (b + 1) for b, f in enumerate(fin)], table, free, nf, bs, B * max_blocks, in_place)


def _check_release(lens, fin, table, free, nf, bs, num_blocks, in_place=False):
    ref = release_ref(lens, fin, table, free, nf, bs, num_blocks)
    L, f, tb, fr, n = _t(lens), _t(fin), _t(table), _t(free), _t([nf])
    status = torch.zeros(1, dtype=I32, device="cuda")
    kw = dict(seq_lens_out=L, num_free_out=n) if in_place else {}
    lo, no = paged_release(L, f, tb, fr, n, bs, num_blocks, status=status, **kw)
    torch.cuda.synchronize()
    assert lo.tolist() == ref[0] and fr.tolist() == ref[1] and no.tolist() == [ref[2]]
    assert bool(status.item() & 1) == ref[3]
    assert tb.tolist() == table


@pytest.mark.parametrize("nf,room", [(3, 0), (3, 2), (3, 9), (-1, 9), (99, 9)])
def test_release_without_room_or_with_bad_values(nf, room):
    lens, fin = [40, 10, 500, 33, 0], [1, 0, 1, 1, 1]
    table = [[0, 1, 77, -7], [3, -7, -7, -7], [4, 5, 6, 7], [8, 9, 10, -7], [-7] * 4]
    _check_release(lens, fin, table, [20, 21, 22] + [-9] * room, nf, 16, 30)


def test_extend_and_release_return_every_block():
    """Random steps with in-place state: the free list and the tables together always hold every block once."""
    g = torch.Generator().manual_seed(0)
    B, bs, num_blocks, max_blocks = 20, 16, 400, 40
    L, nf = torch.zeros(B, dtype=I32, device="cuda"), _t([num_blocks])
    table = torch.full((B, max_blocks), -1, dtype=I32, device="cuda")
    free = torch.randperm(num_blocks, generator=g).to(I32).cuda()
    for step in range(30):
        new = torch.randint(0, 60, (B,), generator=g).to(I32).cuda()
        fin = (torch.rand(B, generator=g) < 0.4).to(I32).cuda()
        paged_extend(L, new, table, free, nf, bs, num_blocks, 2000, seq_lens_out=L, num_free_out=nf)
        held = [-1 - x if x < 0 else x for x in L.tolist()]
        used = [e for b in range(B) for e in table[b, :-(-held[b] // bs)].tolist()]
        assert sorted(used + free[:int(nf)].tolist()) == list(range(num_blocks)), step
        fin |= (L < 0).to(I32)  # what could not be served ends
        paged_release(L, fin, table, free, nf, bs, num_blocks, seq_lens_out=L, num_free_out=nf)
    assert 0 < int(nf) < num_blocks


def test_captured_steps_replay_on_new_lengths():
    B, bs, num_blocks, max_blocks = 9, 16, 300, 30
    L, new = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")
    table = torch.full((B, max_blocks), -1, dtype=I32, device="cuda")
    free, nf = torch.arange(num_blocks, dtype=I32, device="cuda"), _t([num_blocks])
    paged_extend(L, new, table, free, nf, bs, num_blocks, 64)  # first launch outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, _, cu, pos, slots = paged_extend(L, new, table, free, nf, bs, num_blocks, 64, seq_lens_out=L,
                                            num_free_out=nf)
    lens, tb, n = [0] * B, [[-1] * max_blocks for _ in range(B)], num_blocks
    for step in range(4):
        add = [(step * 5 + b * 3) % 8 for b in range(B)]
        new.copy_(_t(add))
        graph.replay()
        torch.cuda.synchronize()
        tb, lens, n, rcu, rpos, rslots, _ = extend_ref(lens, add, tb, list(range(num_blocks)), n, bs, num_blocks, 64)
        assert (L.tolist(), nf.item(), table.tolist()) == (lens, n, tb)
        assert (cu.tolist(), pos.tolist(), slots.tolist()) == (rcu, rpos, rslots)


def test_extend_on_a_named_stream():
    s = torch.cuda.Stream()
    lens, new, table, free, nf = _state(50, 16, 30, 1600, 9, 300, 100)
    _check_extend(lens, new, table, free, nf, 16, 1600, sum(new), stream=s)


def test_refusals():
    ok = dict(seq_lens=_t([1, 2]), new_lens=_t([1, 1]), block_table=_t([[0, 1], [2, 3]]), free_blocks=_t([4, 5]),
              num_free=_t([2]), block_size=16, num_blocks=6, max_tokens=2)

    def call(**kw):
        a = dict(ok, **kw)
        return paged_extend(a.pop("seq_lens"), a.pop("new_lens"), **a)

    call()
    for kw, err in [(dict(seq_lens=torch.zeros(2, dtype=I32)), ValueError), (dict(new_lens=_t([1])), ValueError),
                    (dict(new_lens=_t([1, 1]).long()), TypeError), (dict(block_table=_t([0, 1])), ValueError),
                    (dict(block_table=_t([[0, 1], [2, 3]]).t()), ValueError), (dict(num_free=_t([1, 2])), ValueError),
                    (dict(free_blocks=torch.zeros(2, dtype=I32)), ValueError), (dict(block_size=0), AttnError),
                    (dict(num_blocks=0), AttnError), (dict(max_tokens=-1), AttnError),
                    (dict(num_blocks=2 ** 28), AttnError), (dict(positions=_t([1])), ValueError),
                    (dict(status=torch.zeros(1, device="cuda")), TypeError)]:
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(ValueError):
        paged_release(_t([1, 2]), _t([1]), ok["block_table"], ok["free_blocks"], ok["num_free"], 16, 6)
