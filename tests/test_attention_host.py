"""Refusals of attention, the cache append and the calls on pages: every check happens on
the host, before any launch (CPU)."""
import ctypes

import pytest

import ternary_quantized_moe_amd as tq
from ternary_quantized_moe_amd.binding import KvPoolC

ARG, FORMAT, SHAPE, SPACE = -1, -2, -3, -6
BF16, F16, F32, E4M3 = 0, 1, 2, 3
Q, K, V, Y, LSE, S, WS = (0x10000000 * i for i in range(1, 8))


def message():
    return tq.lib().moe_last_error().decode()


def test_prefill_refusals():
    L = tq.lib()

    def rc(type=BF16, q=Q, n=100, H=8, qt=1024, qh=128, k=K, v=V, m=100, Hk=2, kt=256, kh=128, vt=256, vh=128, D=128, s=S,
           ks=None, seqs=3, scale=0.1, y=Y, lse=LSE, ws=None, wn=0):
        return L.moe_attention_prefill(type, q, n, H, qt, qh, k, v, m, Hk, kt, kh, vt, vh, D, s, ks, seqs, 1, scale, y, lse,
                                       ws, wn, None)
    assert rc(type=F32) == FORMAT and rc(type=E4M3) == FORMAT and rc(type=9) == FORMAT
    for bad in (dict(D=96), dict(D=512), dict(D=0), dict(H=7), dict(H=0), dict(Hk=0), dict(Hk=3), dict(H=8192, Hk=2),
                dict(n=-1), dict(m=-1), dict(n=1 << 31), dict(m=1 << 31), dict(seqs=-1), dict(seqs=(1 << 22) + 1)):
        assert rc(**bad) == SHAPE, bad
    for x in ("qt", "qh", "kt", "kh", "vt", "vh"):
        assert rc(**{x: 132}) == SHAPE and rc(**{x: 120}) == SHAPE and rc(**{x: -128}) == SHAPE and rc(**{x: 1 << 25}) == SHAPE
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert rc(scale=scale) == ARG
    for x in ("q", "k", "v", "s", "y"):
        assert rc(**{x: None}) == ARG
    for x in ("q", "k", "v", "y"):
        assert rc(**{x: 0x90000008}) == ARG
    assert rc(lse=LSE + 2) == ARG and rc(s=S + 1) == ARG and rc(ks=S + 2) == ARG
    assert rc(y=Q) == ARG and rc(y=K + 16) == ARG and rc(y=V - 16) == ARG and rc(lse=Y) == ARG and rc(y=S - 64) == ARG
    assert "overlap" in message()
    assert rc(n=0) == 0 and rc(seqs=0) == 0 and rc(n=0, q=None, y=None) == 0
    need = L.moe_attention_prefill_workspace_bytes(5, 10000, 1, 8, 2, 128)
    assert need > 0
    few = dict(n=5, m=10000, seqs=1, ks=S + 64, wn=need, ws=WS)
    assert rc(**{**few, "ws": None}) == ARG and rc(**{**few, "ws": WS + 16}) == ARG and rc(**{**few, "wn": need - 1}) == SPACE
    assert rc(**{**few, "y": WS + 1024}) == ARG


def test_prefill_workspace():
    f = tq.lib().moe_attention_prefill_workspace_bytes
    assert f(0, 100, 1, 8, 2, 64) == 0 and f(100, 100, 0, 8, 2, 64) == 0 and f(16384, 16384, 1, 16, 4, 128) == 0
    assert f(5, 100, 1, 8, 2, 64) == 0 and f(1 << 30, 1 << 30, 1, 8, 2, 64) == 0
    for bad in ((-1, 1, 1, 8, 2, 64), (1, -1, 1, 8, 2, 64), (1, 1, -1, 8, 2, 64), (1, 1, 1, 8, 3, 64), (1, 1, 1, 8, 2, 65)):
        assert f(*bad) == -1


def test_decode_refusals():
    L = tq.lib()
    need = L.moe_attention_decode_workspace_bytes(4, 8, 2, 128)
    assert need > 0 and L.moe_attention_decode_workspace_bytes(4, 512, 512, 64) == 0
    for bad in ((-1, 8, 2, 64), (1 << 16, 8, 2, 64), (4, 8, 3, 64), (4, 8, 2, 100)):
        assert L.moe_attention_decode_workspace_bytes(*bad) == -1

    def rc(type=BF16, q=Q, B=4, H=8, qt=1024, qh=128, ct=BF16, k=K, v=V, ks=None, vs=None, pages=50, Hk=2, P=16, D=128,
           tab=S, width=10, lens=S + 0x1000, scale=0.1, y=Y, lse=LSE, ws=WS, wn=need):
        return L.moe_attention_decode(type, q, B, H, qt, qh, ct, k, v, ks, vs, pages, Hk, P, D, tab, width, lens, scale, y,
                                      lse, ws, wn, None)
    assert rc(type=F32) == FORMAT and rc(ct=F16) == FORMAT and rc(ct=F32) == FORMAT and rc(type=F16) == FORMAT
    for bad in (dict(D=32), dict(H=9), dict(B=-1), dict(B=65536), dict(P=0), dict(P=24), dict(P=8192), dict(P=-16),
                dict(pages=0), dict(pages=1 << 31), dict(width=-1), dict(qt=1000 + 4), dict(qh=64)):
        assert rc(**bad) == SHAPE, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(tab=None), dict(lens=None), dict(y=None), dict(ws=None),
                dict(k=K + 8), dict(v=V + 2), dict(q=Q + 4), dict(y=Y + 8), dict(tab=S + 2), dict(lens=S + 3), dict(lse=LSE + 1),
                dict(ws=WS + 128), dict(scale=0.0), dict(ks=LSE, vs=LSE + 0x10000), dict(ct=E4M3), dict(ct=E4M3, ks=0x90000000),
                dict(y=K + 4096), dict(ws=Y), dict(lse=S), dict(y=Q), dict(lse=S + 0x1000)):
        assert rc(**bad) == ARG, bad
    assert rc(wn=need - 1) == SPACE
    assert rc(B=0) == 0


def test_append_refusals():
    L = tq.lib()
    QO, KO, R, P_, F = (0x90000000 + 0x10000000 * i for i in range(5))

    def rc(type=BF16, q=Q, qt=1024, qh=128, H=8, k=K, kt=256, kh=128, v=V, vt=256, vh=128, T=5, ct=BF16, kc=Y, vc=LSE, ks=None,
           vs=None, pages=50, Hk=2, P=16, D=128, tab=S, rows=4, width=10, row=R, pos=P_, f=F, rot=128, qo=QO, qot=1024, qoh=128,
           ko=KO, kot=256, koh=128):
        return L.moe_kv_append(type, q, qt, qh, H, k, kt, kh, v, vt, vh, T, ct, kc, vc, ks, vs, pages, Hk, P, D, tab, rows,
                               width, row, pos, f, rot, 0, qo, qot, qoh, ko, kot, koh, None)
    assert rc(type=F32) == FORMAT and rc(ct=F16) == FORMAT
    for bad in (dict(D=80), dict(H=3), dict(T=-1), dict(T=1 << 31), dict(rows=0), dict(rot=24), dict(rot=144), dict(rot=-16),
                dict(P=3), dict(pages=0), dict(width=-1), dict(kt=130), dict(qot=64), dict(koh=64), dict(qot=512, qoh=128)):
        assert rc(**bad) == SHAPE, bad
    for bad in (dict(f=None), dict(rot=0), dict(q=None), dict(qo=None), dict(rot=0, f=None), dict(k=None), dict(v=None),
                dict(kc=None), dict(row=None), dict(pos=None), dict(tab=None), dict(ct=E4M3), dict(ks=WS, vs=WS + 0x100000),
                dict(k=K + 8), dict(qo=QO + 8), dict(f=F + 2), dict(row=R + 1), dict(kc=LSE), dict(kc=K), dict(vc=S), dict(qo=K),
                dict(qo=KO), dict(qo=Q + 16), dict(ko=V), dict(ko=K + 256), dict(qo=P_), dict(ko=F - 16)):
        assert rc(**bad) == ARG, bad
    # q, k and v side by side in one matrix's rows: in place is fine, into each other is not
    row = dict(q=Q, qt=1536, k=Q + 2048, kt=1536, v=Q + 2560, vt=1536, qot=1536, kot=1536)
    assert rc(**row, qo=Q + 256, ko=Q + 2048) == ARG and rc(**row, qo=Q, ko=Q + 2560) == ARG
    assert rc(**row, qo=Q, ko=Q) == ARG
    assert rc(T=0) == 0


def test_pages_refusals():
    L = tq.lib()
    need = L.moe_kv_pages_workspace_bytes(4, 50)
    assert need > 0 and L.moe_kv_pages_workspace_bytes(-1, 5) == -1 and L.moe_kv_pages_workspace_bytes(4, 0) == -1
    T, LEN, REF, ASK, ST = Q, K, V, Y, LSE
    pool = (KvPoolC * 2)(KvPoolC(0xA0000000, 3, 4096), KvPoolC(0xB0000000, 3, 64))

    def reserve(t=T, R=4, w=10, ln=LEN, ref=REF, n=50, P=16, ask=ASK, st=ST, ws=WS, wn=need):
        return L.moe_kv_reserve(t, R, w, ln, ref, n, P, ask, st, ws, wn, None)

    def fork(t=T, R=4, w=10, ln=LEN, ref=REF, n=50, P=16, ask=ASK, st=ST, ws=WS, wn=need, pools=pool, np=2):
        return L.moe_kv_fork(t, R, w, ln, ref, n, P, ask, pools, np, st, ws, wn, None)

    def free(t=T, R=4, w=10, ln=LEN, ref=REF, n=50, P=16, ask=ASK):
        return L.moe_kv_free(t, R, w, ln, ref, n, P, ask, None)

    def compact(t=T, R=4, w=10, ln=LEN, ref=REF, n=50, P=16, nt=ASK, nr=ST, lv=S, ws=WS, wn=need, pools=pool, np=2):
        return L.moe_kv_compact(t, R, w, ln, ref, n, P, pools, np, nt, nr, lv, ws, wn, None)
    for f in (reserve, fork, free, compact):
        for bad in (dict(R=-1), dict(R=1 << 24), dict(w=0), dict(w=-5), dict(n=0), dict(n=1 << 31), dict(P=0), dict(P=48)):
            assert f(**bad) == SHAPE, (f, bad)
        for bad in (dict(t=None), dict(ln=None), dict(ref=None), dict(t=T + 2), dict(ref=REF + 1)):
            assert f(**bad) == ARG, (f, bad)
        assert f(R=0) == 0
    for f in (reserve, fork, compact):
        assert f(ws=None) == ARG and f(ws=WS + 64) == ARG and f(wn=need - 1) == SPACE
    for f in (reserve, fork, free):
        assert f(ask=None) == ARG and f(ask=ASK + 2) == ARG and f(ask=REF) == ARG and f(ln=T) == ARG
    for f in (reserve, fork):
        assert f(st=None) == ARG and f(st=ASK) == ARG and f(st=WS) == ARG
    for f in (fork, compact):
        assert f(np=9) == ARG and f(np=-1) == ARG and f(pools=None) == ARG
        for p, rc in (((0xA0000000, 0, 64), SHAPE), ((0xA0000000, 1, 66), SHAPE), ((0xA0000000, 1, 0), SHAPE),
                      ((None, 1, 64), ARG), ((0xA0000002, 1, 64), ARG), ((T, 1, 64), ARG), ((WS, 1, 64), ARG), ((0xB0000100, 1, 64), ARG)):
            assert f(pools=(KvPoolC * 2)(KvPoolC(*p), pool[1])) == rc, (f, p)
    assert compact(nt=None) == ARG and compact(nr=None) == ARG and compact(lv=None) == ARG and compact(nr=LEN) == ARG
    assert compact(nt=T + 16) == ARG and compact(nr=T) == ARG and compact(lv=REF) == ARG and compact(nt=REF) == ARG
    copy = lambda src=ASK, dst=ST, n=5, pages=50, pools=pool, np=2: L.moe_kv_copy_pages(pools, np, pages, src, dst, n, None)
    assert copy(n=-1) == SHAPE and copy(pages=0) == SHAPE and copy(src=None) == ARG and copy(dst=ST + 1) == ARG
    assert copy(src=0xA0000010) == ARG and copy(np=9) == ARG and copy(n=0) == 0 and copy(np=0) == 0


def test_shapes_and_devices_are_refused_by_the_binding():
    torch = pytest.importorskip("torch")
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: tq.attention_prefill(q, q, q, torch.zeros(2, dtype=torch.int32)),
                 lambda: tq.kv_reserve(torch.zeros((2, 2), dtype=torch.int32), *(torch.zeros(2, dtype=torch.int32) for _ in range(3)), 4),
                 lambda: tq.kv_append(q, q, q, q, q, q, q), lambda: tq.attention_decode(q, q, q, q, q),
                 lambda: tq.kv_copy_pages([q], torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(tq.MoeError, match="device tensor is wanted"):
            call()
    assert ctypes.sizeof(KvPoolC) == 24
