"""Argument checks of the sequence, window and draft-check calls: every one is refused on the
host before any work is enqueued, so no GPU is needed."""
import ctypes

import pytest

import quantized_gated_delta_amd as Q
from quantized_gated_delta_amd import sq as S

P = 0x7F0000000000   # 256-byte aligned, never dereferenced on the host
BIG = 1 << 40


def refused(status, text, fn, *args, **kw):
    with pytest.raises(Q.SQError) as e:
        fn(*args, **kw)
    assert e.value.status == status, (e.value.status, e.value.text)
    assert text in e.value.text, e.value.text


def desc(**kw):
    d = dict(n_seq=2, n_tokens=100, n_heads=4, d=128, gate=Q.SQ_GATE_GDN, in_dtype=Q.SQ_BF16, y_dtype=Q.SQ_BF16, n_key_heads=2)
    d.update(kw)
    return Q.seq_desc(**d)


def forward(dsc=None, stream=0, **kw):
    a = dict(cu=P, q=P, k=P, v=P, beta=P, g=P, S0=P, y=P, S_out=P, save=None, work=P, save_bytes=0, work_bytes=BIG)
    a.update(kw)
    Q.sq_chunk_forward(dsc or desc(), stream=stream, **a)


def backward(dsc=None, stream=0, **kw):
    a = dict(cu=P, q=P, k=P, v=P, beta=P, g=P, dy=P, dS_out=P, save=P, dq=P, dk=P, dv=P, dbeta=P, dg=P, dS0=P, work=P, save_bytes=BIG,
             work_bytes=BIG)
    a.update(kw)
    Q.sq_chunk_backward(dsc or desc(), stream=stream, **a)


BAD_DESC = [
    (dict(n_seq=-1), Q.SQ_EINVAL, "n_seq"), (dict(n_tokens=-1), Q.SQ_EINVAL, "n_tokens"), (dict(n_heads=0, n_key_heads=1), Q.SQ_EINVAL, "n_heads"),
    (dict(n_key_heads=3), Q.SQ_EINVAL, "divisor"), (dict(n_key_heads=-2), Q.SQ_EINVAL, "divisor"), (dict(d=96), Q.SQ_EUNSUPPORTED, "64 or 128"),
    (dict(gate=2), Q.SQ_EINVAL, "gate"), (dict(in_dtype=2), Q.SQ_EINVAL, "in_dtype"), (dict(y_dtype=-1), Q.SQ_EINVAL, "y_dtype"),
    (dict(n_tokens=1 << 31), Q.SQ_EUNSUPPORTED, "n_tokens"), (dict(n_tokens=(1 << 31) - 70, n_heads=100), Q.SQ_EUNSUPPORTED, "grid"),
    (dict(q_stride=2 * 128 - 8), Q.SQ_EINVAL, "q_stride"), (dict(k_stride=2 * 128 + 4), Q.SQ_EINVAL, "k_stride"),
    (dict(v_stride=4 * 128 + 1), Q.SQ_EINVAL, "v_stride"), (dict(v_stride=-1024), Q.SQ_EINVAL, "v_stride"),
    (dict(in_dtype=Q.SQ_F32, v_stride=4 * 128 + 2), Q.SQ_EINVAL, "v_stride"), (dict(q_stride=1 << 60), Q.SQ_EINVAL, "q_stride"),
]


@pytest.mark.parametrize("change,status,text", BAD_DESC, ids=lambda x: str(x) if isinstance(x, dict) else "")
def test_descriptor(change, status, text):
    for call in (Q.sq_chunk_bytes, forward, backward):
        refused(status, text, call, desc(**change))


def test_descriptor_null_and_unequal_dims():
    out = ctypes.c_size_t()
    assert Q.lib().sq_chunk_bytes(None, ctypes.byref(out), None) == Q.SQ_EINVAL and "desc is NULL" in Q.sq_last_error()
    d = desc()
    d.d_v = 64
    refused(Q.SQ_EUNSUPPORTED, "d_k must equal", Q.sq_chunk_bytes, d)
    assert Q.lib().sq_chunk_bytes(ctypes.byref(desc()), None, None) == Q.SQ_EINVAL


def test_bytes_grow_with_the_batch_alone():
    """One buffer of the largest batch serves every smaller one."""
    for gate in (Q.SQ_GATE_GDN, Q.SQ_GATE_KDA):
        for dt in (Q.SQ_F32, Q.SQ_BF16):
            last = (0, 0)
            for n_tokens in (0, 1, 63, 64, 65, 1000, 5000):
                for n_seq in (1, 2, 9):
                    now = Q.sq_chunk_bytes(desc(gate=gate, in_dtype=dt, n_tokens=n_tokens, n_seq=n_seq), train=True)
                    assert now[0] >= Q.sq_chunk_bytes(desc(gate=gate, in_dtype=dt, n_tokens=n_tokens, n_seq=n_seq))
                    if n_seq == 9:
                        assert now >= last
                        last = now
    assert Q.sq_chunk_bytes(desc(n_seq=0, n_tokens=0)) == 0


POINTERS = [("cu", 1, "4-byte"), ("beta", 1, "2-byte"), ("g", 1, "2-byte")] + [(x, 8, "16-byte") for x in ("q", "k", "v")]


@pytest.mark.parametrize("name,off,text", POINTERS + [("y", 2, "16-byte"), ("S0", 4, "16-byte"), ("S_out", 4, "16-byte"), ("work", 16, "256-byte")])
def test_forward_pointers(name, off, text):
    refused(Q.SQ_EINVAL, "%s is not %s" % (name, text), forward, **{name: P + off})
    if name not in ("S0", "S_out"):
        refused(Q.SQ_EINVAL, "%s is NULL" % name, forward, **{name: None})


@pytest.mark.parametrize("name,off,text", POINTERS + [(x, 8, "16-byte") for x in ("dy", "dq", "dk", "dv", "dS_out", "dS0")] +
                         [("dbeta", 1, "2-byte"), ("dg", 1, "2-byte"), ("work", 128, "256-byte"), ("save", 64, "256-byte")])
def test_backward_pointers(name, off, text):
    refused(Q.SQ_EINVAL, "%s is not %s" % (name, text), backward, **{name: P + off})
    if name not in ("dS_out", "dS0"):
        refused(Q.SQ_EINVAL, "%s is NULL" % name, backward, **{name: None})


def test_gates_per_channel_are_read_in_vectors():
    d = desc(gate=Q.SQ_GATE_KDA)
    refused(Q.SQ_EINVAL, "g is not 16-byte", forward, d, g=P + 8)
    refused(Q.SQ_EINVAL, "dg is not 16-byte", backward, d, dg=P + 8)
    d = desc(in_dtype=Q.SQ_F32)
    refused(Q.SQ_EINVAL, "beta is not 4-byte", forward, d, beta=P + 2)


def test_buffers_too_small():
    work, save = Q.sq_chunk_bytes(desc(), train=True)
    refused(Q.SQ_ENOMEM, "work has", forward, work_bytes=Q.sq_chunk_bytes(desc()) - 1)
    refused(Q.SQ_ENOMEM, "save has", forward, save=P, save_bytes=save - 1)
    refused(Q.SQ_EINVAL, "save is not 256-byte", forward, save=P + 16, save_bytes=save)
    refused(Q.SQ_ENOMEM, "save has", backward, save_bytes=save - 1)
    refused(Q.SQ_ENOMEM, "work has", backward, work_bytes=work - 1)


def test_nothing_to_do():
    """No sequence: a no-op whatever the pointers."""
    nothing = dict(cu=None, q=None, k=None, v=None, beta=None, g=None, save=None, work=None, work_bytes=0)
    forward(desc(n_seq=0, n_tokens=0), S0=None, y=None, S_out=None, **nothing)
    backward(desc(n_seq=0, n_tokens=0), dy=None, dq=None, dk=None, dv=None, dbeta=None, dg=None, dS_out=None, dS0=None, **nothing)


def pool(gate=Q.SQ_GATE_GDN):
    bits = [6, 4, 8, 16]
    n = Q.sq_pool_bytes(8, 4, 128, 128, bits, gate)
    return Q.sq_pool_create(8, 4, 128, 128, bits, gate, P, n)


def window(handle, **kw):
    a = dict(slot_idx=P, n=3, length=4, lens=None, n_key_heads=2, q=P, k=P, v=P, beta=P, g=P, y=P, S_out=P, in_dtype=Q.SQ_BF16, y_dtype=Q.SQ_BF16,
             stream=0)
    a.update(kw)
    Q.sq_window_update(handle, **a)


def f32_window(**kw):
    a = dict(state=P, n_slots=8, n_heads=4, n_key_heads=2, d_k=128, d_v=128, gate=0, slot_idx=P, n=3, length=4, lens=None, q=P, k=P, v=P, beta=P, g=P,
             y=P, S_out=P, in_dtype=Q.SQ_BF16, y_dtype=Q.SQ_BF16, stream=0)
    a.update(kw)
    Q.sq_f32_window_update(**a)


BAD_WINDOW = [
    (dict(length=0), "length"), (dict(length=17), "length"), (dict(n_key_heads=3), "divisor"), (dict(n_key_heads=0), "divisor"),
    (dict(in_dtype=5), "in_dtype"), (dict(y_dtype=5), "y_dtype"), (dict(y=None, S_out=None), "both NULL"), (dict(lens=P + 2), "lens"),
    (dict(q=None), "q is NULL"), (dict(k=None), "k is NULL"), (dict(v=P + 4), "v is not"), (dict(beta=None), "beta is NULL"), (dict(g=P + 8), "g is not"),
    (dict(y=P + 2), "y is not"), (dict(S_out=P + 4), "S_out is not"), (dict(slot_idx=None), "slot_idx"), (dict(n=-1), "n must be"), (dict(n=9), "n_slots"),
]


@pytest.mark.parametrize("change,text", BAD_WINDOW, ids=lambda x: str(x) if isinstance(x, dict) else "")
def test_window_refusals(change, text):
    h = pool()
    try:
        refused(Q.SQ_EINVAL, text, window, h, **change)
    finally:
        Q.sq_pool_destroy(h)
    refused(Q.SQ_EINVAL, text, f32_window, **change)


def test_window_shapes_and_no_op():
    refused(Q.SQ_EINVAL, "pool is NULL", window, None)
    refused(Q.SQ_EINVAL, "state_pool is NULL", f32_window, state=None)
    refused(Q.SQ_EINVAL, "gate", f32_window, gate=7)
    refused(Q.SQ_EUNSUPPORTED, "d_k must equal", f32_window, d_v=64)
    refused(Q.SQ_EUNSUPPORTED, "64 or 128", f32_window, d_k=32, d_v=32)
    refused(Q.SQ_EINVAL, "n_slots", f32_window, n_slots=0)
    refused(Q.SQ_EINVAL, "n_heads", f32_window, n_heads=0)
    f32_window(n=0, slot_idx=None, q=None, k=None)
    h = pool()
    window(h, n=0, slot_idx=None, k=None)
    Q.sq_pool_destroy(h)


def verify(**kw):
    a = dict(n=3, m=4, vocab=1000, target=P, target_stride=0, draft=P, draft_stride=0, tokens=P, lens=None, accept_u=P, sample_e=P, temperature=1.0,
             accepted=P, next_token=P, work=P, work_bytes=BIG, logits_dtype=Q.SQ_BF16, stream=0)
    a.update(kw)
    Q.sq_verify_draft(**a)


BAD_VERIFY = [
    (dict(n=-1), Q.SQ_EINVAL, "n must be"), (dict(m=0), Q.SQ_EINVAL, "m must be"), (dict(m=33), Q.SQ_EINVAL, "m must be"),
    (dict(vocab=0), Q.SQ_EINVAL, "vocab"), (dict(vocab=0x7FFFFFFF), Q.SQ_EINVAL, "vocab"), (dict(logits_dtype=9), Q.SQ_EINVAL, "logits_dtype"),
    (dict(temperature=-0.5), Q.SQ_EINVAL, "temperature"), (dict(temperature=float("nan")), Q.SQ_EINVAL, "temperature"),
    (dict(temperature=float("inf")), Q.SQ_EINVAL, "temperature"), (dict(temperature=1e-42), Q.SQ_EINVAL, "temperature"),
    (dict(target_stride=999), Q.SQ_EINVAL, "stride"), (dict(draft_stride=-1), Q.SQ_EINVAL, "stride"), (dict(target_stride=1 << 60), Q.SQ_EINVAL, "stride"),
    (dict(n=30000), Q.SQ_EUNSUPPORTED, "rows"), (dict(target=None), Q.SQ_EINVAL, "target is NULL"), (dict(target=P + 1), Q.SQ_EINVAL, "target is not"),
    (dict(draft=P + 1), Q.SQ_EINVAL, "draft is not"), (dict(tokens=None), Q.SQ_EINVAL, "tokens is NULL"), (dict(lens=P + 2), Q.SQ_EINVAL, "lens is not"),
    (dict(accept_u=None), Q.SQ_EINVAL, "accept_u is NULL"), (dict(sample_e=None), Q.SQ_EINVAL, "sample_e is NULL"),
    (dict(accepted=None), Q.SQ_EINVAL, "accepted is NULL"), (dict(next_token=P + 1), Q.SQ_EINVAL, "next is not"),
    (dict(work=None), Q.SQ_EINVAL, "work is NULL"), (dict(work=P + 8), Q.SQ_EINVAL, "work is not"), (dict(work_bytes=10), Q.SQ_ENOMEM, "work has"),
]


@pytest.mark.parametrize("change,status,text", BAD_VERIFY, ids=lambda x: str(x) if isinstance(x, dict) else "")
def test_verify_refusals(change, status, text):
    refused(status, text, verify, **change)


def test_verify_no_op_and_bytes():
    verify(n=0, target=None, tokens=None, work=None, work_bytes=0)
    assert Q.sq_verify_bytes(0, 1) == 0
    assert Q.sq_verify_bytes(64, 8) >= Q.sq_verify_bytes(64, 4) >= Q.sq_verify_bytes(1, 4) > 0
    assert Q.lib().sq_verify_bytes(1, 1, None) == Q.SQ_EINVAL


def test_new_calls_are_declared_with_their_errors():
    from tests.test_abi import PAGES, _declaration_comments
    com = _declaration_comments()
    for name in ("sq_chunk_bytes", "sq_chunk_forward", "sq_chunk_backward", "sq_window_update", "sq_f32_window_update", "sq_verify_bytes", "sq_verify_draft"):
        assert name in com, name
        assert "SQ_EINVAL" in com[name] or "rrors" in com[name], name
    for name in ("sq_chunk_forward", "sq_window_update", "sq_f32_window_update"):
        assert any(p in com[name] for p in PAGES), name


def test_limits_match_the_header():
    text = open(S.HEADER).read()
    assert "#define SQ_WINDOW_MAX %d\n" % Q.SQ_WINDOW_MAX in text
    assert "#define SQ_DRAFT_MAX %d\n" % Q.SQ_DRAFT_MAX in text
