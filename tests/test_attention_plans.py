"""Plans of the attention layer on the host: what a call hands to the library, with the library's entry points
replaced by recorders and CPU tensors that stand for device memory (no GPU: nothing is launched)."""
import threading

import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding as B


class OnDevice(torch.Tensor):
    """A CPU tensor that says it lies in the memory of device `index`."""
    index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


def dev(t, index=0):
    t = t.as_subclass(OnDevice)
    t.index = index
    return t


@pytest.fixture(scope="module", autouse=True)
def library():
    from delta_rule_recurrent_gated_gb300 import build
    build.build()
    return B.load()


def here(plan, stream=7):
    """A plan of the CPU as one of device 0, on a stream of the test's."""
    plan._index, plan._stream = 0, lambda: stream
    return plan


def norm(T=3, Hq=4, Hk=2, d=64):
    return here(B.HeadNormRope(2, T, Hq, Hk, d, device="cpu"))


def packed(heads, T=3, d=64, width=8):
    return dev(torch.zeros(2, T, width, d, dtype=torch.bfloat16)[:, :, :heads])


def plain(heads, T=3, d=64):
    return dev(torch.zeros(2, T, heads, d, dtype=torch.bfloat16))


def tables(rows, d=64):
    return [dev(torch.zeros(rows, d // 2)) for _ in range(2)]


class Cache(B.KvCache):
    """A cache of the CPU as one of device 0."""

    def _at(self, device):
        super()._at(device)
        here(self)


def cache(other=None):
    """`other`: the buffer that lies on another device."""
    kinds = [torch.zeros(8, 2, 16, 64, dtype=torch.int8) for _ in range(2)] + [torch.zeros(8, 2) for _ in range(2)]
    return Cache(8, 2, 64, page=16, buffers=[dev(t, int(i == other)) for i, t in enumerate(kinds)], device="cpu")


def places():
    return dev(torch.zeros(2, 4, dtype=torch.int32)), dev(torch.zeros(2, dtype=torch.int32))


def in_a_thread(f):
    out = []
    t = threading.Thread(target=lambda: out.append(f()))
    t.start()
    t.join(30)
    assert out, "the other thread's call did not return"


def test_two_threads_hand_over_their_own_layouts():
    """A call that another thread's comes between (the library is called without the interpreter's lock)."""
    p, seen = norm(), []

    def entry(ref, *rest):
        d = ref._obj
        if not seen:
            seen.append(None)
            in_a_thread(lambda: p.forward(packed(4), packed(2, width=6), None, None, *tables(9)))
        seen.append((d.ld_q, d.ld_k, d.ld_oq, d.ld_ok, d.table_rows))
        return 0

    p._fwd = entry
    p.forward(plain(4), plain(2), None, None, *tables(5), yq=packed(4, width=5))
    assert seen[1:] == [(512, 384, 256, 128, 9), (256, 128, 320, 128, 5)]

    p, seen = norm(), []

    def entry(ref, *rest):  # noqa: F811
        d = ref._obj
        if not seen:
            seen.append(None)
            in_a_thread(lambda: p.forward(packed(4), packed(2, width=6), None, None, *tables(9)))
        seen.append((d.ld_q, d.ld_k, d.ld_oq, d.ld_ok, d.table_rows))
        return 0

    p._bwd = p._fwd = entry
    p.backward(plain(4), plain(2), None, None, *tables(5), plain(4), plain(2))
    assert seen[1:] == [(512, 384, 256, 128, 9), (256, 128, 256, 128, 5)]


def test_two_threads_hand_over_their_own_queries():
    a, seen = here(B.CacheAttention(cache(), 2, 3, 4)), []

    def entry(c, s, ref, *rest):
        if not seen:
            seen.append(None)
            in_a_thread(lambda: a.forward(packed(4), *places(), o=plain(4)))
        seen.append(ref._obj.ld_q)
        return 0

    a._attn = entry
    a.forward(plain(4), *places(), o=plain(4))
    assert seen[1:] == [512, 256]


def test_a_refused_call_leaves_the_gradient_its_workspace():
    """A row distance that the library refuses is that call's alone."""
    p, got = norm(), []
    wide = dev(torch.zeros(2 * 3 * 258 + 8, dtype=torch.bfloat16).as_strided((2, 3, 4, 64), (3 * 258, 258, 64, 1)))
    with pytest.raises(B.DrError) as e:
        p.forward(wide, plain(2), None, None, *tables(5))
    assert e.value.code == B.DR_ERR_ALIGNMENT
    need = int(B.load().dr_norm_rope_workspace_bytes(norm()._ref))
    p._bwd = lambda *a: got.append(a[-3:-1]) or 0
    p.backward(plain(4), plain(2), None, None, *tables(5), plain(4), plain(2))
    (address, size), = got
    assert need > 0 and size == need and address


def test_tensors_of_another_device_are_refused():
    p, c = norm(), cache()
    a = here(B.CacheAttention(c, 2, 3, 4))
    ran = []
    p._fwd = p._bwd = a._attn = c._write = c._read = lambda *x: ran.append(x) or 0
    good = [plain(4), plain(2), dev(torch.zeros(64)), dev(torch.zeros(64)), *tables(5)]
    outs = dict(yq=plain(4), yk=plain(2), positions=dev(torch.zeros(2, 3, dtype=torch.int32)), start=places()[1])
    p.forward(*good, **outs)
    for i in range(6):
        with pytest.raises(ValueError):
            p.forward(*good[:i], dev(good[i].clone(), 1), *good[i + 1:])
    for n, t in outs.items():
        with pytest.raises(ValueError):
            p.forward(*good, **{n: dev(t.clone(), 1)})
    for i in (0, 1):
        dy = [plain(4), plain(2)]
        dy[i] = dev(dy[i].clone(), 1)
        with pytest.raises(ValueError):
            p.backward(*good, *dy)
    table, lens = places()
    for q, t, n, extra in ((plain(4), table, lens, {}), (plain(4), table, lens, dict(counts=lens))):
        a.forward(q, t, n, o=plain(4), **extra)
        args = [q, t, n]
        for i in range(3):
            with pytest.raises(ValueError):
                a.forward(*args[:i], dev(args[i].clone(), 1), *args[i + 1:], o=plain(4), **extra)
    with pytest.raises(ValueError):
        a.forward(plain(4), table, lens, o=dev(plain(4).clone(), 1))
    k = plain(2)
    for args in ((dev(k.clone(), 1), k), (k, dev(k.clone(), 1))):
        with pytest.raises(ValueError):
            c.write(*args, table, lens)
    with pytest.raises(ValueError):
        c.read(table, lens, lens, 3, k=dev(k.clone(), 1), v=k)
    assert len(ran) == 3
    on_host = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        a.forward(on_host, table, lens, o=plain(4))


def test_a_cache_of_another_device_is_refused():
    for i in range(4):
        with pytest.raises(ValueError):
            cache(other=i)


def test_a_plan_runs_on_its_own_device_only(monkeypatch):
    """The default stream's handle names the stream of whichever device is current."""
    p = B.HeadNormRope(2, 3, 4, 2, 64, device="cpu")
    p._index, p._raw, p._current = 0, lambda i: 7, lambda: 0
    assert p._stream() == 7
    p._current = lambda: 1
    with pytest.raises(ValueError):
        p._stream()


def test_streams_and_threads_have_workspaces_of_their_own():
    """Calls that may run at the same time, or whose kernels may interleave, share no workspace."""
    a, p, used = here(B.CacheAttention(cache(), 2, 3, 4)), norm(), []
    a._attn = lambda *x: used.append(x[-3:-1]) or 0
    p._bwd = lambda *x: used.append(x[-3:-1]) or 0

    def attend():
        a.forward(plain(4), *places(), o=plain(4))

    def gradient():
        p.backward(plain(4), plain(2), None, None, *tables(5), plain(4), plain(2))

    for plan, call in ((a, attend), (p, gradient)):
        used.clear()
        call()
        call()
        here(plan, stream=8)
        call()
        other_thread = threading.Thread(target=call)
        other_thread.start()
        other_thread.join(30)
        here(plan, stream=7)
        call()
        (first, size), second, other, thread, back = used
        assert second == back == (first, size)
        addresses = sorted({first, other[0], thread[0]})
        assert len(addresses) == 3 and all(y - x >= size for x, y in zip(addresses, addresses[1:]))
        assert other[1] == thread[1] == size


def test_plans_over_one_cache_share_its_workspaces():
    """A program with prompts of any length makes a plan for each; their workspaces do not add up."""
    c, used = cache(), []
    for T in (1, 2, 40, 41, 80, 200):
        a = here(B.CacheAttention(c, 2, T, 4))
        a._attn = lambda *x: used.append(x[-3:-1]) or 0
        a.forward(plain(4, T=T), *places(), o=plain(4, T=T))
        assert used[-1][1] == int(B.load().dr_cache_attn_workspace_bytes(c._ref, a._ref, 2, T))
    assert len(set(used)) == 2  # one for each of the two kernels
