"""The plan of a step's requests -- pages, starts, positions, slots -- against a loop over the requests."""
import concurrent.futures
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tf():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ulysses_sequence_attention_tf_gb300 import binding, build
    build.build()
    binding.lib()
    yield binding
    torch.cuda.synchronize()
    assert binding.device_status() == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def by_hand(table, lens, new, free, span, page, rows):
    """Everything as lists; and whether something was out of range."""
    table, free, out = [list(r) for r in table], list(free), list(lens)
    cap, room = len(free), len(table[0]) * page if table else 0
    head, count = span
    bad = not (0 <= head < cap and 0 <= count <= cap)
    back_room = 0 if bad else cap - count
    if bad:
        head = count = 0
    before = list(free)
    taken = tokens = 0
    open_, starts, positions, slots, back = True, [0], [], [], []
    for n, (length, more) in enumerate(zip(lens, new)):
        if not 0 <= length <= room or (more > 0 and length + more > room):
            bad = True
        elif more < 0:
            back += table[n][: -(-length // page)]
            out[n] = 0
        elif open_:
            had = -(-length // page)
            need = -(-(length + more) // page) - had
            if taken + need > count or tokens + more > rows:
                open_ = False
            else:
                for x in range(need):
                    table[n][had + x] = before[(head + taken + x) % cap]
                taken, tokens = taken + need, tokens + more
                for at in range(length, length + more):
                    positions.append(at)
                    slots.append(table[n][at // page] * page + at % page)
                out[n] = length + more
        starts.append(tokens)
    if len(back) > back_room:
        bad, back = True, back[:back_room]
    for x, id_ in enumerate(back):
        free[(head + count + x) % cap] = id_
    fill = rows - len(positions)
    return dict(page_table=table, free=free, lens=out, starts=starts, positions=positions + [0] * fill, slots=slots + [-1] * fill,
                span=[(head + taken) % cap, count - taken + len(back)]), bad


def run(tf, table, lens, new, free, span, page, rows, **kw):
    """Twice: the same call again gives the same."""
    args = [i32(table) if table else torch.zeros((0, 4), dtype=torch.int32, device="cuda"), i32(lens), i32(new), i32(free), i32(span)]
    want, bad = by_hand(table, lens, new, free, span, page, rows)
    for _ in range(2):
        p = tf.kv_plan(*args, page_size=page, rows=rows, **kw)
        got = dict(page_table=args[0], free=args[3], **p._asdict())
        for name, x in want.items():
            assert got[name].dtype == torch.int32 and got[name].tolist() == x, name
        assert args[1].tolist() == list(lens) and args[4].tolist() == list(span)
    assert tf.device_status(clear=True) == (8 if bad else 0)
    return p


def case(rng, N, page, most, *, ended=0.2, tokens=40, spare=5, tight=0):
    lens = [rng.choice([0, rng.randint(0, most * page), page * rng.randint(0, most)]) for _ in range(N)]
    new = [-rng.randint(1, 5) if rng.random() < ended else min(rng.choice([0, 1, 1, rng.randint(0, tokens)]), most * page - n) for n in lens]
    up = lambda n: -(-n // page)  # noqa: E731
    held = sum(up(n) for n in lens)
    need = sum(up(n + t) - up(n) for n, t in zip(lens, new) if t > 0)
    pages = max(1, held + max(0, need + spare - tight))
    ids = list(range(pages))
    rng.shuffle(ids)
    table, at = [], 0
    for n in lens:
        table.append(ids[at:at + up(n)] + [-7] * (most - up(n)))
        at += up(n)
    head, free = rng.randrange(pages), [-9] * pages
    for x, id_ in enumerate(ids[held:]):
        free[(head + x) % pages] = id_
    rows = sum(max(0, t) for t in new)
    return table, lens, new, free, [head, pages - held], page, rows


@pytest.mark.parametrize("N,page,most", [(1, 16, 4), (2, 16, 1), (31, 32, 8), (33, 16, 6), (64, 128, 5), (1000, 16, 20), (1025, 64, 4), (3000, 16, 9)])
@pytest.mark.parametrize("seed", range(3))
def test_random_requests(tf, N, page, most, seed):
    args = case(random.Random(100 * N + seed), N, page, most)
    run(tf, *args)


@pytest.mark.parametrize("seed", range(6))
def test_pages_or_rows_run_out(tf, seed):
    rng = random.Random(seed)
    *args, rows = case(rng, 100, 16, 8, tight=rng.randint(6, 60))
    run(tf, *args, rows)
    run(tf, *args, rows // 2)
    run(tf, *args, 0)
    run(tf, *args, rows + 3000)


def test_most_requests(tf):
    rng = random.Random(8)
    run(tf, *case(rng, 8192, 16, 3))
    run(tf, *case(rng, 8192, 16, 3, tight=4000))


def test_prompts_over_many_blocks(tf):
    """More rows than one block of threads takes, and rows behind the last."""
    args = case(random.Random(2), 200, 16, 128, tokens=2000, ended=0.1)
    assert args[-1] > 20000
    run(tf, *args[:-1], args[-1] + 1500)


def test_no_requests(tf):
    run(tf, [], [], [], [3, 1, 2], [1, 2], 16, 5)


def test_lengths_of_zero_and_ends(tf):
    # nothing new; a page filled to its end; one more token; a whole row of pages; an ended request without tokens
    table = [[4, -1, -1], [5, -1, -1], [6, -1, -1], [-1, -1, -1], [-1, -1, -1]]
    run(tf, table, [7, 16, 15, 0, 0], [0, 1, 1, 48, -1], [0, 1, 2, 3, 7, 8, 9, 10], [6, 5], 16, 50)


@pytest.mark.parametrize("lens,new", [([-1, 5], [3, 3]), ([65, 5], [0, 3]), ([2 ** 31 - 1, 5], [2 ** 31 - 1, 3]), ([60, 5], [5, 3]),
                                      ([5, 5], [2 ** 31 - 1, 3]), ([-2 ** 31, 5], [-1, 3]), ([70, 5], [-1, 3])])
def test_lengths_out_of_range_are_left_out(tf, lens, new):
    p = run(tf, [[1, 2, 3, 4], [5, 6, 7, 8]], lens, new, list(range(16)), [3, 4], 16, 10)
    assert p.starts.tolist() == [0, 0, 3] and p.lens.tolist() == [lens[0], 8]


@pytest.mark.parametrize("span", [[-1, 3], [8, 3], [0, 9], [0, -1], [2 ** 31 - 1, 2 ** 31 - 1]])
def test_spans_out_of_range_give_nothing(tf, span):
    table = [[1, 2], [3, 4], [5, 6]]
    p = run(tf, table, [16, 5, 20], [1, 3, -1], list(range(8)), span, 16, 10)
    assert p.starts.tolist() == [0, 0, 0, 0]


def test_more_pages_given_back_than_fit(tf):
    run(tf, [[1, 2, 3], [4, 5, 6]], [40, 40], [-1, -1], list(range(6)), [4, 2], 16, 4)


@pytest.mark.parametrize("page,bad", [(16, -1), (16, 2 ** 27), (128, 2 ** 31 - 1), (64, -2 ** 31)])
@pytest.mark.parametrize("fresh", [False, True])
def test_rows_on_pages_out_of_range_have_no_slot(tf, page, bad, fresh):
    """The page that a request has, or the one that it takes; the largest that has slots beside it."""
    largest = 2 ** 31 // page - 1
    lens = [0, 0] if fresh else [2, 2]
    table, free = ([[-7], [-7]], [bad, largest]) if fresh else ([[bad], [largest]], [3, 4])
    t = [i32(table), i32(lens), i32([3, 3]), i32(free), i32([0, 2])]
    p = tf.kv_plan(*t, page_size=page, rows=8)
    at = lens[0]
    assert p.slots.tolist() == [-1] * 3 + [largest * page + at + x for x in range(3)] + [-1] * 2
    assert p.starts.tolist() == [0, 3, 6] and p.lens.tolist() == [at + 3] * 2
    assert tf.device_status(clear=True) == 8


def test_given_outputs_strides_streams_and_graphs(tf):
    args = case(random.Random(5), 40, 16, 6)
    table, lens, new, free, span, page, rows = args
    wide = torch.full((40, 11), -3, dtype=torch.int32, device="cuda")
    wide[:, :6] = i32(table)
    t = [wide[:, :6], i32(lens), i32(new), i32(free), i32(span)]
    outs = {n: torch.full((s,), -5, dtype=torch.int32, device="cuda") for n, s in
            (("lens_out", 40), ("starts", 41), ("positions", rows), ("slots", rows), ("span_out", 2))}
    want, _ = by_hand(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = tf.kv_plan(*t, page_size=page, rows=rows, stream=side, **outs)
    torch.cuda.current_stream().wait_stream(side)
    assert p.lens is outs["lens_out"] and p.span is outs["span_out"]
    assert p.slots.tolist() == want["slots"] and t[0].tolist() == want["page_table"] and bool((wide[:, 6:] == -3).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tf.kv_plan(*t, page_size=page, rows=rows, **outs)
    # a step: what the plan gave is where the next one starts
    for step in range(3):
        now = [t[0].tolist(), t[1].tolist(), t[2].tolist(), t[3].tolist(), t[4].tolist()]
        graph.replay()
        want, bad = by_hand(*now, page, rows)
        assert not bad and outs["positions"].tolist() == want["positions"] and outs["slots"].tolist() == want["slots"]
        assert t[0].tolist() == want["page_table"] and t[3].tolist() == want["free"] and outs["span_out"].tolist() == want["span"]
        t[1].copy_(outs["lens_out"])
        t[4].copy_(outs["span_out"])
        t[2].copy_(torch.where(t[1] > 60, -1, 1))
        assert rows >= 40


def test_calls_of_several_threads(tf):
    """Large and small calls at once, each on its own stream: one's shared memory is not what the other asked for."""
    cases = [case(random.Random(7), 8000, 16, 3), case(random.Random(8), 3, 16, 3)] * 2
    wants = [by_hand(*c)[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    inputs = [[i32(x) for x in c[:5]] for c in cases]
    torch.cuda.synchronize()

    def calls(i):
        for _ in range(200):
            p = tf.kv_plan(*inputs[i], page_size=cases[i][5], rows=cases[i][6], stream=streams[i])
        streams[i].synchronize()
        return p

    with concurrent.futures.ThreadPoolExecutor(len(cases)) as pool:
        got = list(pool.map(calls, range(len(cases))))
    for p, want in zip(got, wants):
        assert p.slots.tolist() == want["slots"] and p.lens.tolist() == want["lens"]


def test_refusals(tf):
    good = [torch.zeros((3, 4), dtype=torch.int32, device="cuda"), i32([0] * 3), i32([0] * 3), i32([0] * 6), i32([0, 0])]
    for i, x in [(0, good[0].long()), (0, good[0].cpu()), (0, good[0].t()), (1, i32([0] * 4)), (1, None), (2, good[2].float()), (3, good[0]),
                 (4, i32([0] * 3)), (4, None)]:
        with pytest.raises(ValueError):
            tf.kv_plan(*[x if j == i else g for j, g in enumerate(good)], page_size=16, rows=4)
    for kw in (dict(rows=-1), dict(rows=2 ** 40), dict(rows=4, starts=i32([0] * 3)), dict(rows=4, slots=i32([0] * 5))):
        with pytest.raises(ValueError):
            tf.kv_plan(*good, page_size=16, **kw)
    for kw in (dict(page_size=8), dict(page_size=16, lens_out=good[1]), dict(page_size=16, span_out=good[4])):
        with pytest.raises(tf.TfUlyssesError):
            tf.kv_plan(*good, rows=4, **kw)
