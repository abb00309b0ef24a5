"""PagedKV, the binding's handle of a paged cache: whichever way one is made, its C
structure holds the addresses of its own tensors. Stand-ins for CUDA tensors, so
that this runs without a GPU; nothing is launched."""
import copy
import pickle

import pytest
import torch

from speech_encoder_attention_b200 import attn

CUDA = torch.device("cuda", 0)


class Fake:
    """What PagedKV looks at in a contiguous CUDA tensor."""
    is_cuda = True
    places = iter(range(1 << 20, 1 << 40, 1 << 20))

    def __init__(self, *shape, dtype=torch.int32, device=CUDA):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device
        self.at = next(Fake.places)

    def stride(self):
        return (self.shape[-1], 1)[-len(self.shape):]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at

    def __deepcopy__(self, memo):
        return Fake(*self.shape, dtype=self.dtype, device=self.device)

    def __reduce__(self):
        return _fake, (tuple(self.shape), self.dtype)


def _fake(shape, dtype):
    return Fake(*shape, dtype=dtype)


def pool(rows=64, cols=128):
    return Fake(rows, cols, dtype=torch.float16)


def cache(batch=2, per_seq=3):
    return attn.PagedKV(pool(), pool(), Fake(batch, per_seq), Fake(batch), 16, 2)


def addresses(c):
    return c.k.ptr, c.v.ptr, c.table, c.kv_lens


def check(c):
    assert addresses(c.c) == (c.k.at, c.v.at, c.table.at, c.lens.at)
    assert (c.c.num_pages, c.c.page_size, c.c.pages_per_seq, c.c.n_kv_heads) == (
        c.k.shape[0] // c.page_size, c.page_size, c.table.shape[1], c.n_kv_heads)
    assert (c.batch, c.slots, c.device) == (c.table.shape[0], c.table.shape[1] * c.page_size, CUDA)


def test_replaced_tensors_reach_the_c_structure():
    c = cache()
    check(c)
    before = addresses(c.c)
    for new in (dict(lens=Fake(2)), dict(table=Fake(2, 5)), dict(k=pool(), v=pool()), dict(page_size=32),
                dict(n_kv_heads=1), dict(k=pool(96), v=pool(96), table=Fake(4, 1), lens=Fake(4)), {}):
        got = c._replace(**new)
        assert type(got) is attn.PagedKV and all(getattr(got, name) is x for name, x in new.items())
        check(got)
    assert addresses(c.c) == before


@pytest.mark.parametrize("bad", [
    dict(lens=Fake(3)), dict(lens=Fake(2, dtype=torch.int64)), dict(table=Fake(3, 3)), dict(table=Fake(6)),
    dict(k=pool(48)), dict(v=pool(cols=64)), dict(page_size=24), dict(page_size=128), dict(n_kv_heads=4),
    dict(lens=Fake(2, device=torch.device("cuda", 1))), dict(batch=1), dict(c=None), dict(slots=16), dict(no=1),
])
def test_replacements_are_checked(bad):
    with pytest.raises(ValueError):
        cache()._replace(**bad)


def test_copies_are_made_of_their_own_tensors():
    c = cache()
    same = copy.copy(c)
    check(same)
    assert same.lens is c.lens and addresses(same.c) == addresses(c.c)
    for other in (copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        check(other)
        assert not set(addresses(other.c)) & set(addresses(c.c))


def test_a_cache_is_not_made_of_its_fields():
    c = cache()
    with pytest.raises(TypeError):
        attn.PagedKV._make(tuple(c))
    with pytest.raises(AttributeError):
        c.lens = Fake(2)
