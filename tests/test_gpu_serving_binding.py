"""GPU tests of what the serving calls' Python side does around the library."""
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    import quantized_attention_08_b200 as s
    s.load_library()
    return s


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class NoTruth:
    def __bool__(self):
        raise RuntimeError("neither")


def test_flags_without_a_truth_value(sage):
    """The exception of the flag's own, and no call with a flag left unset."""
    c = sage.SageKVCache.allocate(3, 2, 16, 64, "16")
    q = torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
    for kw in (dict(causal=NoTruth()), dict(return_lse=NoTruth())):
        with pytest.raises(RuntimeError, match="neither"):
            sage.sage_attn_decode_paged(q, c, ints([[0, 1]]), ints([20]), 32, **kw)
    # two-element tensors have no truth value either
    with pytest.raises(RuntimeError, match="more than one value"):
        sage.sage_attn_decode_paged(q, c, ints([[0, 1]]), ints([20]), 32, causal=ints([0, 1]))


@pytest.mark.parametrize("fmt", ["16", "8+8"])
def test_means_of_no_request(sage, fmt):
    """Tokens whose request has no mean are skipped, also where no request has one."""
    c = sage.SageKVCache.allocate(2, 2, 16, 64, fmt)
    x = torch.ones(2, 3, 64, dtype=torch.float16, device="cuda")
    for B in (0, 1):
        mean = torch.ones(B, 2, 64, device="cuda")
        sage.sage_kv_append(x, x, ints([0, 5, 9]), c, mean_k=mean, seq_ids=ints([B, -1, B + 7]))
        assert not any(bool(t.any()) for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None), B


def test_other_threads_run_while_the_queue_is_full(sage):
    """A call whose launch waits for room in the stream's queue does not hold the
    interpreter: behind a kernel of half a second or more, thousands of calls
    block, and this thread goes on meanwhile."""
    c = sage.SageKVCache.allocate(2, 1, 16, 64, "16")
    x, slot = torch.ones(1, 1, 64, dtype=torch.float16, device="cuda"), ints([3])
    q, pos, inv = x[None], ints([[1]]), torch.ones(32, device="cuda")
    lens, table, ws = ints([4]), ints([[0]]), torch.empty(256, dtype=torch.uint8, device="cuda")
    out = tuple(ints([0] * n) for n in (1, 2, 1, 1, 1, 1))
    o = torch.empty_like(q)
    calls = [lambda: sage.sage_kv_append(x, x, slot, c),
             lambda: sage.sage_rope_axes(q, None, pos, inv, [32], q_out=o),
             lambda: sage.sage_kv_slots(ints_lens, one, free, used, table, page_size=16, T=1, out=out),
             lambda: sage.sage_attn_decode_paged(q, c, table, lens, 4, o=o, workspace=ws)]
    ints_lens, one, free, used = ints([0]), ints([1]), ints([0, 1]), ints([0])
    for call in calls:
        call()
        torch.cuda.synchronize()
        done = []

        def work():
            torch.cuda._sleep(1_000_000_000)  # clock cycles: half a second at 1965 MHz
            at = time.perf_counter()
            for _ in range(3000):
                call()
            done.append(time.perf_counter() - at)

        t = threading.Thread(target=work)
        t.start()
        longest, last = 0.0, time.perf_counter()
        while not done:
            time.sleep(0.001)
            now = time.perf_counter()
            longest, last = max(longest, now - last), now
        t.join()
        torch.cuda.synchronize()
        assert done[0] > 0.3, "the queue did not fill"
        assert longest < 0.15, (longest, done)


def test_kept_lengths_keep_no_tokens(sage):
    """The results that go on to the next step hold no memory of the step's tokens."""
    T = 20000
    got = sage.sage_kv_slots(ints([3, 9]), ints([7, 2]), ints([4, 5, 6]), ints([0]), ints([[0, -1], [1, -1]]),
                             page_size=16, T=T)
    assert [len(t) for t in got] == [2, 3, T, T, T, 1]
    lens, cu, slots, pos, ids, used = got
    assert max(t.untyped_storage().nbytes() for t in (lens, cu, used)) <= 64
    assert lens.tolist() == [10, 11] and cu.tolist() == [0, 7, 9] and used.tolist() == [0]
    assert slots[:9].tolist() == list(range(3, 10)) + [25, 26] and slots[9:].unique().tolist() == [-1]
    assert pos[:9].tolist() == list(range(3, 10)) + [9, 10] and ids[:9].tolist() == [0] * 7 + [1] * 2
    for a in (lens, slots, used):  # parts of one allocation stay apart
        a.fill_(77)
    assert cu.tolist() == [0, 7, 9] and pos[:2].tolist() == [3, 4] and ids[-1].item() == -1
