"""GPU tests of what the serving calls' Python side does around the library."""
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
