"""A prompt through the model with a block-causal mask, in float64: block by block through the oracle's layer (a block
of M positions sees everything before it and itself), each block's keys and values joining the prefix."""
import numpy as np

from oracle import focus_oracle as fo


def prompt_forward(shape, model, tokens, mask_block, store=None):
    """(K/V [L, 2, Hkv, P, d], residual rows after the last layer [P, D]) of one prompt."""
    store = store or (lambda x: x)
    L, hkv, d, P = shape.n_layers, shape.n_kv_heads, shape.head_dim, len(tokens)
    keys = ("attn_norm", "wqkv", "wo", "mlp_norm", "wgate", "wup", "wdown")
    lws = [{k: fo._f64(model[k][l]) for k in keys} for l in range(L)]
    embed = fo._f64(model["embed"])
    kv = np.zeros((L, 2, hkv, P, d))
    hidden = np.zeros((P, embed.shape[1]))
    for p in range(0, P, mask_block):
        e = min(P, p + mask_block)
        x = embed[np.asarray(tokens[p:e])]
        for l in range(L):
            ck, cv = np.zeros((hkv, e - p, d)), np.zeros((hkv, e - p, d))
            x, _ = fo.layer_forward(x, lws[l], shape, np.arange(p, e), np.arange(e - p), kv[l, 0, :, :p], kv[l, 1, :, :p],
                                    ck, cv, store)
            kv[l, 0, :, p:e], kv[l, 1, :, p:e] = ck, cv
        hidden[p:e] = x
    return kv, hidden


def cached(pool, table_row, n):
    """K/V [L, 2, Hkv, n, d] of a request's first n positions, from the page pool."""
    S = pool.shape[4]
    pages = [int(p) for p in table_row[: -(-n // S)]]
    a = fo._f64(pool[pages])                                     # [pages, L, 2, Hkv, S, d]
    return a.transpose(1, 2, 3, 0, 4, 5).reshape(*a.shape[1:4], -1, a.shape[5])[:, :, :, :n]
