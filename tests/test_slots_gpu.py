"""drs_map_slots against a plain implementation (Python integers): every
output, the table and the ring, exactly, with everything that the call must
not write filled with a sentinel."""
import numpy as np
import pytest
import torch

from gpu_util import drs

pytestmark = pytest.mark.gpu

FILL = -77


def reference(lens, new, held, table, block, ring, state, capacity):
    table, ring = table.copy(), ring.copy()
    requests, widest = table.shape
    size, (head, tail) = len(ring), (int(state[0]), int(state[1]))
    avail = min(max(tail - head, 0), size)
    asked = given = taken = lacking = tokens = 0
    cu, now_held = [], []
    request, position, slot = np.full(capacity, -1), np.zeros(capacity, np.int64), np.full(capacity, -1)
    old_ring = ring.copy()
    for b in range(requests):
        length, fresh = max(int(lens[b]), 0), max(int(new[b]), 0)
        have = min(max(int(held[b]), 0), widest)
        want = -(-(length + fresh) // block)
        need = min(want, widest)
        take = max(need - have, 0)
        served = asked + take <= avail
        now = need if served else min(need, have)
        if served:
            for i in range(take):
                table[b, have + i] = old_ring[(head + asked + i) % size]
            taken += take
        asked += take
        for i in range(need, have):
            ring[(tail + given) % size] = table[b, i]
            given += 1
        lacking += want - now
        now_held.append(now)
        cu.append(min(tokens, capacity))
        upto = min(tokens + fresh, capacity)
        if upto > tokens:
            pos = length + np.arange(upto - tokens, dtype=np.int64)
            request[tokens:upto] = b
            position[tokens:upto] = np.minimum(pos, 2**31 - 1)
            col = pos // block
            ok = col < now
            slot[tokens:upto][ok] = table[b][col[ok]].astype(np.int64) * block + pos[ok] % block
        tokens += fresh
    cu.append(min(tokens, capacity))
    return (np.array(cu), request, position, slot, np.array(now_held, np.int64).reshape(requests),
            np.array([head + taken, tail + given]), np.array([lacking]), table, ring)


def state_of(seed, requests, most_len, most_new, block, widest=None, spare=None, pad=0, held_extra=0.3):
    """A consistent cache: distinct block ids in the table and the ring."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most_len + 1, requests).astype(np.int32)
    new = rng.integers(0, most_new + 1, requests).astype(np.int32)
    ended = rng.random(requests) < 0.15
    extra = (rng.random(requests) < held_extra) * rng.integers(0, 4, requests)
    held = -(-lens // block) + extra
    lens[ended], new[ended] = 0, 0
    if widest is None:
        widest = max(1, int(max(held.max(initial=0), (-(-(lens + new) // block)).max(initial=0))) + 2)
    held = np.minimum(held, widest).astype(np.int32)
    want = np.minimum(-(-(lens + new) // block), widest)
    needed = int(np.maximum(want - held, 0).sum())
    spare = needed + 5 if spare is None else spare
    pool = rng.permutation(int(held.sum()) + spare + 3).astype(np.int32)
    table = np.full((requests, widest + pad), FILL, np.int32)
    at = 0
    for b in range(requests):
        table[b, : held[b]] = pool[at:at + held[b]]
        at += held[b]
    size = len(pool)
    head = int(rng.integers(0, 5 * size))
    ring = np.full(size, FILL, np.int32)
    ring[(head + np.arange(spare)) % size] = pool[at:at + spare]
    return lens, new, held, table, widest, block, ring, np.array([head, head + spare], np.int64)


def check(case, capacity, in_place=False, where=None):
    lens, new, held, table, widest, block, ring, state = case
    lib = drs()
    dev = lambda a: torch.as_tensor(np.ascontiguousarray(a)).cuda()
    full, g_ring, g_held, g_state = dev(table), dev(ring), dev(held), dev(state)
    requests = len(lens)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (torch.full((requests + 1,), FILL, **i32), torch.full((capacity,), FILL, **i32),
           torch.full((capacity,), FILL, **i32), torch.full((capacity,), FILL, dtype=torch.int64, device="cuda"),
           g_held if in_place else torch.full((requests,), FILL, **i32),
           g_state if in_place else torch.full((2,), FILL, dtype=torch.int64, device="cuda"), torch.full((1,), FILL, **i32))
    lib.map_slots(dev(lens), dev(new), g_held, full[:, :widest], block, g_ring, g_state, capacity, out=out)
    ref = reference(lens, new, held, table[:, :widest], block, ring, state, capacity)
    got = [t.cpu().numpy() for t in out] + [full[:, :widest].cpu().numpy(), g_ring.cpu().numpy()]
    names = ("cu", "request", "position", "slot", "held", "state", "lacking", "table", "ring")
    for name, g, r in zip(names, got, ref):
        assert np.array_equal(g, r), (where, name)
    assert np.array_equal(full[:, widest:].cpu().numpy(), table[:, widest:]), (where, "padding")
    return ref


@pytest.mark.parametrize("requests", [0, 1, 2, 31, 32, 33, 255, 1000, 1024, 1025, 5000])
@pytest.mark.parametrize("block", [1, 16, 24])
def test_requests_and_blocks(requests, block):
    case = state_of(requests + block, requests, 200, 6, block)
    total = int(case[1].sum())
    for capacity in (total, total + 7):
        check(case, capacity, where=(requests, block, capacity))


@pytest.mark.parametrize("block", [16, 64, 128, 1000])
def test_long_prompts(block):
    """Requests of one token beside prompts of thousands; tokens cut at the capacity."""
    case = state_of(block, 40, 3000, 5, block)
    case[0][[3, 17]] = 0
    case[1][[3, 17, 39]] = [9000, 1, 20011]
    lens, new = case[0], case[1]
    need = -(-(lens + new) // block)
    widest = int(need.max()) + 1
    rng = np.random.default_rng(1)
    held = np.minimum(case[2], widest)
    spare = int(np.maximum(need - held, 0).sum()) + 1
    pool = rng.permutation(int(held.sum()) + spare).astype(np.int32)
    table = np.full((40, widest), FILL, np.int32)
    at = 0
    for b in range(40):
        table[b, : held[b]] = pool[at:at + held[b]]
        at += held[b]
    ring = np.full(len(pool), FILL, np.int32)
    ring[np.arange(spare)] = pool[at:]
    case = (lens, new, held, table, widest, block, ring, np.array([0, spare], np.int64))
    total = int(new.sum())
    for capacity in (total, total - 1000, 1, 0, total + 5000):
        check(case, capacity, where=(block, capacity))


@pytest.mark.parametrize("spare", [0, 1, 2, 10, 60])
def test_ring_that_runs_out(spare):
    """Requests are served in order while the ring lasts; the others keep what
    they hold and their tokens beyond it get no slot."""
    for seed in range(4):
        case = state_of(seed, 50, 100, 40, 8, spare=spare, held_extra=0.0)
        ref = check(case, int(case[1].sum()), where=(spare, seed))
        assert ref[6][0] > 0 and (ref[3][: ref[0][-1]] == -1).any()


def test_table_that_is_too_narrow():
    case = state_of(2, 60, 400, 50, 16, widest=8, pad=3)
    ref = check(case, int(case[1].sum()))
    assert ref[6][0] > 0


def test_in_place_counts_and_odd_inputs():
    """held and ring_state updated in place; negative lengths and counts, a
    count of held blocks past the table, counters past 32 bits."""
    for requests, seed in ((7, 1), (3000, 2)):
        case = list(state_of(seed, requests, 300, 9, 16, pad=1))
        check(case, int(case[1].sum()), in_place=True, where=requests)
        case[7] = case[7] + (len(case[6]) << 33)
        check(case, int(case[1].sum()), in_place=True, where="large counters")
    lens, new, held = (np.array(a, np.int32) for a in ([-5, 10, 3, 2**31 - 10], [4, -3, 2, 9], [-2, 1, 1, 0]))
    table = np.arange(4 * 6, dtype=np.int32).reshape(4, 6) + 100
    case = (lens, new, held, table, 6, 16, np.arange(32, dtype=np.int32), np.array([3, 20], np.int64))
    check(case, 40, where="negative")
    held[:] = [9, 9, 9, 9]
    check((lens, new, held, table, 6, 16, np.full(64, 5, np.int32), np.array([0, 0], np.int64)), 40, where="held past the table")
    # counters that make no sense lead nowhere outside the ring
    check((lens, new, np.array([0, 1, 0, 2], np.int32), table, 6, 16, np.arange(7, dtype=np.int32),
           np.array([10, 4], np.int64)), 40, where="tail before head")


def test_block_ids_past_32_bit_slots():
    case = list(state_of(5, 20, 500, 8, 128))
    case[3] = np.where(case[3] >= 0, case[3] + 2**30, case[3]).astype(np.int32)
    case[6] = np.where(case[6] >= 0, case[6] + 2**30, case[6]).astype(np.int32)
    ref = check(case, int(case[1].sum()))
    assert ref[3].max() > 2**36


def test_table_offsets_past_32_bits():
    """Rows of the table 2^22 entries apart, the last ones past 2^32 entries."""
    case = list(state_of(6, 1100, 60, 9, 16, widest=8))
    far = torch.empty(1100 * 2**22, dtype=torch.int32, device="cuda").view(1100, 2**22)[:, :8]
    far.copy_(torch.as_tensor(case[3]))
    dev = lambda a: torch.as_tensor(np.ascontiguousarray(a)).cuda()
    ring, capacity = dev(case[6]), int(case[1].sum())
    out = drs().map_slots(dev(case[0]), dev(case[1]), dev(case[2]), far, 16, ring, dev(case[7]), capacity)
    ref = reference(case[0], case[1], case[2], case[3], 16, case[6], case[7], capacity)
    for got, want in zip(list(out) + [far, ring], ref):
        assert np.array_equal(got.cpu().numpy(), want)


def test_many_requests():
    case = state_of(9, 70001, 40, 3, 16)
    check(case, int(case[1].sum()) + 1)


def test_large_steps_on_another_stream_and_in_a_graph():
    """The two launches of a large step, in place: on a stream of its own,
    then captured and replayed on other lengths."""
    lib = drs()
    case = state_of(21, 900, 300, 40, 16)
    lens, new, held, table, widest, block, ring, state = case
    capacity = int(new.sum()) + 100
    assert capacity > 8192
    dev = lambda a: torch.as_tensor(np.ascontiguousarray(a)).cuda()
    g = [dev(a) for a in (lens, new, held, table, ring, state)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = lib.map_slots(*g[:4], block, g[4], g[5], capacity, stream=side)
    side.synchronize()
    ref = reference(lens, new, held, table, block, ring, state, capacity)
    for got, want in zip(list(out) + [g[3], g[4]], ref):
        assert np.array_equal(got.cpu().numpy(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.map_slots(*g[:4], block, g[4], g[5], capacity)
    for seed in (22, 23):
        other = state_of(seed, 900, 300, 40, 16, widest=widest)
        size = min(len(ring), len(other[6]))
        fresh = list(other[:4]) + [np.resize(other[6], len(ring)), np.array([3, 3 + size // 2])]
        for t, a in zip(g, fresh):
            t.copy_(torch.as_tensor(np.ascontiguousarray(a)))
        graph.replay()
        ref = reference(fresh[0], fresh[1], fresh[2], fresh[3], block, fresh[4], fresh[5], capacity)
        for got, want in zip(list(out) + [g[3], g[4]], ref):
            assert np.array_equal(got.cpu().numpy(), want)


def test_steps_of_a_cache_on_a_captured_graph():
    """Twelve steps, in place, replayed from one graph: lengths grow and
    shrink, requests end and begin, and no block is ever in two places."""
    lib = drs()
    rng = np.random.default_rng(4)
    requests, block, widest, blocks = 24, 8, 20, 24 * 20
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, new = torch.zeros(requests, **i32), torch.zeros(requests, **i32)
    held, table = torch.zeros(requests, **i32), torch.full((requests, widest), FILL, **i32)
    ring = torch.as_tensor(rng.permutation(blocks).astype(np.int32)).cuda()
    state = torch.tensor([0, blocks], dtype=torch.int64, device="cuda")
    out = (torch.zeros(requests + 1, **i32), torch.zeros(512, **i32), torch.zeros(512, **i32),
           torch.zeros(512, dtype=torch.int64, device="cuda"), held, state, torch.zeros(1, **i32))
    graph = torch.cuda.CUDAGraph()
    lib.load()
    with torch.cuda.graph(graph):
        lib.map_slots(lens, new, held, table, block, ring, state, 512, out=out)
    host = [np.zeros(requests, np.int32), np.full((requests, widest), FILL, np.int32), ring.cpu().numpy(),
            np.array([0, blocks], np.int64)]
    length = np.zeros(requests, np.int32)
    for step in range(12):
        fresh = rng.integers(0, 20, requests).astype(np.int32)
        length = np.where(rng.random(requests) < 0.1, 0, length)
        fresh = np.where(length + fresh > widest * block, 0, fresh).astype(np.int32)
        lens.copy_(torch.as_tensor(length.astype(np.int32)))
        new.copy_(torch.as_tensor(fresh))
        graph.replay()
        ref = reference(length, fresh, host[0], host[1], block, host[2], host[3], 512)
        for got, want in zip([t.cpu().numpy() for t in out] + [table.cpu().numpy(), ring.cpu().numpy()], ref):
            assert np.array_equal(got, want), step
        host = [ref[4].astype(np.int32), ref[7], ref[8], ref[5]]
        used = np.concatenate([ref[7][b, : ref[4][b]] for b in range(requests)])
        free = ref[8][np.arange(ref[5][0], ref[5][1]) % blocks]
        assert sorted(np.concatenate([used, free])) == list(range(blocks)), step
        length = np.maximum(length + fresh - rng.integers(0, 4, requests), 0).astype(np.int32)  # refused drafts
