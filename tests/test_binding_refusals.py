"""Tensors of the wrong number of dimensions and numbers that do not fit the C types are refused with
SpecError by the serving calls, not with whatever indexing or packing raises."""
import pytest

torch = pytest.importorskip("torch")
from speculative_decoding_draft_04_gb300 import _lib, build  # noqa: E402

i32, u8 = torch.int32, torch.uint8
st = torch.zeros(4, dtype=i32)


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.fixture
def packed(monkeypatch):
    """Checks that find every tensor in place, so that only the numbers are left."""
    class Checks:
        @staticmethod
        def addresses(dev, *a):
            out = []
            for _, _, dtype, shape in zip(*[iter(a)] * 4):
                out += [0] * (1 if dtype is not None else 2 if shape is None else 3)
            return tuple(out)
    _lib._types()
    monkeypatch.setattr(_lib, "_args", Checks)
    monkeypatch.setattr(_lib, "_raw_stream", lambda device, stream: 0)   # the library refuses infinite scales itself


def tables(seq_len=torch.zeros(2, dtype=i32), page_size=16):
    v = torch.zeros(2, dtype=i32)
    _lib.spec_block_tables(seq_len, None, v, v, v.long(), v, v.view(2, 1), v, v, v, v.long(), v, v, v, st, page_size)


def attention(mask=None, softmax_scale=1.0, k_scale=1.0):
    q = torch.zeros((4, 2, 64))
    cache = torch.zeros((3, 2, 1, 18 * 64), dtype=u8)
    _lib.spec_cache_attention(q, cache, torch.zeros((1, 2), dtype=i32), st[:1], st[:2], q, st, cache, softmax_scale,
                              k_scale, tree_mask=mask)


def append(**scales):
    x = torch.zeros((4, 2, 64))
    _lib.spec_cache_append(x, x, st, torch.zeros((3, 2, 1, 18 * 64), dtype=u8), st, **scales)


def logprobs(top):
    x = torch.zeros((1, 2, 8))
    _lib.spec_logprobs(x, torch.zeros((1, 2), dtype=i32), x[..., 0], x[..., 0], st, st, top_ids=top, top_logprobs=top)


@pytest.mark.parametrize("shape", [(), (4,), (4, 1, 1)])
def test_dimensions_of_a_tree_mask(shape):
    with pytest.raises(_lib.SpecError, match="tree_mask"):
        attention(mask=torch.zeros(shape, dtype=i32))


@pytest.mark.parametrize("shape", [(), (5,), (1, 2), (1, 2, 5, 1)])
def test_dimensions_of_the_alternatives(shape):
    with pytest.raises(_lib.SpecError, match="top_ids"):
        logprobs(torch.zeros(shape, dtype=i32))


@pytest.mark.parametrize("shape", [(), (2, 1)])
def test_dimensions_of_lengths(shape):
    with pytest.raises(_lib.SpecError, match="seq_len"):
        tables(torch.zeros(shape, dtype=i32))


def test_numbers_that_do_not_fit(packed):
    for call in (lambda: tables(page_size=2 ** 31), lambda: tables(page_size=16.5), lambda: tables(page_size=None),
                 lambda: attention(softmax_scale=1e39), lambda: attention(k_scale="1"),
                 lambda: append(k_scale=-1e300), lambda: append(v_scale=None)):
        with pytest.raises(_lib.SpecError):
            call()
