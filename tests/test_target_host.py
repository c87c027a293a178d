"""Host-side refusals and prices of the paged target cache, its attention and
the logit rules: everything the header documents is refused before anything is
enqueued (the pointers below are stand-ins and never dereferenced)."""
import ctypes as C

import pytest

P = 0x100000  # an aligned stand-in
ODD = P + 8


@pytest.fixture(scope="module")
def A():
    from block_diffusion_speculative_tap_gb300 import _abi as A

    return A


def pages(A, **over):
    f = dict(format=A.PAGES_BF16, n_pages=100, page_size=64, n_kv_heads=8, head_dim=128, streams=4, table_cols=32,
             k=P, v=P, k_scale=P, v_scale=P, table=P)
    f.update(over)
    return A.Pages(*[f[n] for n, _ in A.Pages._fields_])


def rows(A, **over):
    f = dict(rows=64, max_rows=16, row_start=P, lens=P, depth=None)
    f.update(over)
    return A.RowsDesc(*[f[n] for n, _ in A.RowsDesc._fields_])


def attend(A, c=None, r=None, nq=32, q=P, q_ld=4096, scale=0.1, window=0, sinks=0, mode=0, mask=None, mask_ld=0,
           out=P, out_ld=4096, ws=P, wsb=1 << 40):
    c, r = c if c is not None else pages(A), r if r is not None else rows(A)
    return A.lib.dflash_page_attention(C.byref(c), C.byref(r), nq, q, q_ld, scale, window, sinks, mode, mask, mask_ld,
                                       out, out_ld, None, ws, wsb, None)


def append(A, c=None, r=None, k=P, k_ld=1024, v=P, v_ld=1024, rope=P, rope_rows=4096, nq=32, q=P, q_ld=4096, qo=P,
           qo_ld=4096):
    c, r = c if c is not None else pages(A), r if r is not None else rows(A)
    return A.lib.dflash_page_append(C.byref(c), C.byref(r), k, k_ld, v, v_ld, rope, rope_rows, nq, q, q_ld, qo, qo_ld,
                                    None, None)


def read(A, c=None, r=None, k=P, k_ld=1024, v=P, v_ld=1024):
    c, r = c if c is not None else pages(A), r if r is not None else rows(A)
    return A.lib.dflash_page_read(C.byref(c), C.byref(r), k, k_ld, v, v_ld, None, None)


BAD_PAGES = [
    (dict(format=2), -1), (dict(head_dim=96), -5), (dict(head_dim=256), -5), (dict(page_size=8), -5),
    (dict(page_size=48), -5), (dict(page_size=256), -5), (dict(n_kv_heads=0), -5), (dict(n_kv_heads=65536), -5),
    (dict(n_pages=0), -1), (dict(streams=-1), -1), (dict(table_cols=0), -1), (dict(table=None), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(k=P + 64), -1), (dict(v=ODD), -1),
    (dict(table_cols=1 << 25), -6), (dict(n_pages=1 << 22), -6),
    (dict(format=1, k_scale=None), -1), (dict(format=1, v_scale=ODD), -1),
]


def test_pages_and_rows_are_refused_by_every_call(A):
    nb = C.c_size_t()
    price = lambda c, r: A.lib.dflash_page_attention_workspace_bytes(C.byref(c), C.byref(r), 32, C.byref(nb))
    calls = [lambda c, r: attend(A, c, r), lambda c, r: append(A, c, r), lambda c, r: read(A, c, r), price]
    for over, code in BAD_PAGES:
        for call in calls:
            got = call(pages(A, **over), rows(A))
            assert got == code, (over, got)
    for over in (dict(rows=-1), dict(max_rows=-1), dict(row_start=None), dict(lens=None), dict(rows=1 << 30)):
        for call in calls:
            assert call(pages(A), rows(A, **over)) == -1, over
    # nothing to do: accepted, nothing enqueued
    for over in (dict(rows=0), dict(max_rows=0)):
        for call in calls:
            assert call(pages(A), rows(A, **over)) == 0, over
    for call in calls:
        assert call(pages(A, streams=0, table=None), rows(A, row_start=None, lens=None)) == 0
    assert A.lib.dflash_page_attention(None, None, 32, P, 4096, 0.1, 0, 0, 0, None, 0, P, 4096, None, P, 1, None) == -1
    assert A.lib.dflash_page_append(None, None, P, 8, P, 8, None, 0, 0, None, 0, None, 0, None, None) == -1
    assert A.lib.dflash_page_read(None, None, P, 8, P, 8, None, None) == -1
    assert A.lib.dflash_page_attention_workspace_bytes(C.byref(pages(A)), C.byref(rows(A)), 32, None) == -1


def test_attention_refusals(A):
    for nq in (0, -8, 12, 8 * 129):
        assert attend(A, nq=nq) == -5, nq
    assert attend(A, r=rows(A, max_rows=1 << 29)) == -5  # 2^29 rows of four heads a kv head
    nan, inf = float("nan"), float("inf")
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=nan), dict(scale=inf), dict(window=-1), dict(sinks=-1),
                dict(mode=3), dict(mode=-1), dict(mode=2), dict(mode=2, mask=P, mask_ld=0),
                dict(mode=2, mask=P + 2, mask_ld=1), dict(q=None), dict(q=ODD), dict(q_ld=4088), dict(q_ld=4100),
                dict(out=None), dict(out=ODD), dict(out_ld=4095)):
        assert attend(A, **bad) == -1, bad
    nb = C.c_size_t()
    assert A.lib.dflash_page_attention_workspace_bytes(C.byref(pages(A)), C.byref(rows(A)), 32, C.byref(nb)) == 0
    assert nb.value > 0
    for bad in (dict(ws=None), dict(ws=ODD), dict(wsb=nb.value - 1)):
        assert attend(A, **bad) == -7, bad


def test_workspace_is_for_split_streams_only(A):
    """A table too short to be split costs no workspace; the price does not grow
    with the rows of a prompt chunk beyond the slices a GPU can hold."""
    nb = C.c_size_t()

    def price(c, r, nq=32):
        assert A.lib.dflash_page_attention_workspace_bytes(C.byref(c), C.byref(r), nq, C.byref(nb)) == 0
        return nb.value

    assert price(pages(A, table_cols=1), rows(A, rows=4, max_rows=1)) == 0
    assert price(pages(A), rows(A, rows=0)) == 0
    big = price(pages(A), rows(A, rows=4 * 4096, max_rows=4096))
    assert big == price(pages(A), rows(A, rows=4 * 65536, max_rows=65536)) < 1 << 27


def test_append_and_read_refusals(A):
    for bad in (dict(rope=None), dict(rope=None, rope_rows=0), dict(rope=ODD), dict(rope_rows=0), dict(nq=0),
                dict(nq=-1), dict(q=None), dict(qo=None), dict(k=None), dict(k=ODD), dict(k_ld=1016), dict(k_ld=1028),
                dict(v=ODD), dict(v_ld=0), dict(q_ld=4088), dict(qo=ODD), dict(qo_ld=4100)):
        assert append(A, **bad) == -1, bad
    for bad in (dict(k=None), dict(k=ODD), dict(k_ld=1016), dict(v=None), dict(v_ld=1028)):
        assert read(A, **bad) == -1, bad


def test_token_count_refusals(A):
    f = A.lib.dflash_token_counts
    for args in ((-1, 4096, P, P, None, 16, 64, 0), (4, 4, P, P, None, 16, 64, 0), (4, 4092, P, P, None, 16, 64, 0),
                 (4, 4096, None, P, None, 16, 64, 0), (4, 4096, P, None, None, 16, 64, 0),
                 (4, 4096, ODD, P, None, 16, 64, 0), (4, 4096, P, P, None, 0, 64, 0), (4, 4096, P, P, None, 16, 65, 0),
                 (4, 4096, P, P, P, 0, -1, 0), (4, 4096, P, P, None, 16, 64, 2), (4, 4096, P, P, P, 0, (1 << 38) + 1, 0)):
        assert f(*args, None) == -1, args
    assert f(0, 4096, P, P, P, 0, 64, 1, None) == 0
    assert f(4, 4096, P, P, P, 0, 0, 1, None) == 0


def test_logit_rule_refusals(A):
    def rules(**over):
        f = dict(counts=P, tokens=P, node_mask=None, mask_ld=0, n_bias=0, repetition=P, frequency=P, presence=P,
                 bias_start=None, bias_ids=None, bias_vals=None, grammar=None)
        f.update(over)
        return A.Rules(*[f[n] for n, _ in A.Rules._fields_])

    def call(S=4, N=16, V=4096, x=P, out=P, **over):
        u = rules(**over)
        return A.lib.dflash_logit_rules(S, N, V, x, C.byref(u), out, None)

    for bad in (dict(S=-1), dict(N=-1), dict(N=1025), dict(V=4), dict(V=4092), dict(x=None), dict(x=ODD),
                dict(out=None), dict(out=ODD), dict(counts=None), dict(counts=None, tokens=None), dict(counts=ODD),
                dict(counts=None, repetition=None, frequency=None, presence=None), dict(node_mask=P, mask_ld=0),
                dict(tokens=None, node_mask=P, mask_ld=1), dict(bias_start=P), dict(bias_ids=P, bias_vals=P),
                dict(n_bias=-1), dict(grammar=P + 2)):
        assert call(**bad) == -1, bad
    assert A.lib.dflash_logit_rules(4, 16, 4096, P, None, P, None) == -1
    assert call(S=0) == 0 and call(N=0) == 0
