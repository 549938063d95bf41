"""Float64 oracle of the target model's side of a round: row planning, the paged
cache's writes, attention over it, and the adjustment of the target rows.

Each function is the definition of the call of the same name, one request and one
row at a time, in numpy.  Tokens, pages and slots are whole numbers and have to be
equal; attention also returns what the error bound of a float32 evaluation needs.
"""
import numpy as np


def plan_rows(length, advance, rows, held, free_state, free_ring, block_table, page, max_rows):
    """Returns a dict of all outputs, with the updated copies of block_table and free_ring;
    `detail` is 0 or the detail code of a refused step."""
    B = len(length)
    cap, width = len(free_ring), block_table.shape[1]
    table, ring = block_table.copy(), free_ring.copy()
    head, count = int(free_state[0]), int(free_state[1])
    base = [int(n) + int(a) for n, a in zip(length, advance)]
    need = [-(-(x + int(r)) // page) for x, r in zip(base, rows)]
    out = dict(length=np.array(length, np.int32), held=np.array(held, np.int32),
               free_state=np.array(free_state, np.int32), row_offset=np.zeros(B + 1, np.int32),
               row_request=np.full(max_rows, -1, np.int32), position=np.full(max_rows, -1, np.int32),
               slot=np.full(max_rows, -1, np.int64), block_table=table, free_ring=ring, detail=0)
    take = [max(0, n - int(h)) for n, h in zip(need, held)]
    give = [max(0, int(h) - n) for n, h in zip(need, held)]
    bad = any(length[b] < 0 or advance[b] < 0 or rows[b] < 0 or held[b] < 0 or held[b] > width
              or base[b] > int(held[b]) * page for b in range(B))
    if bad or not 0 <= head < cap or not 0 <= count <= cap:
        return dict(out, detail=1)
    if any(base[b] + int(rows[b]) > width * page for b in range(B)):
        return dict(out, detail=2)
    if sum(take) > count:
        return dict(out, detail=3)
    if count + sum(give) > cap:
        return dict(out, detail=1)
    if int(np.sum(rows)) > max_rows:
        return dict(out, detail=4)
    first, tail, i = head, head + count, 0
    for b in range(B):
        for j in range(int(held[b]), need[b]):
            table[b, j] = free_ring[first % cap]
            first += 1
        for j in range(need[b], int(held[b])):
            ring[tail % cap] = block_table[b, j]
            tail += 1
        out["row_offset"][b] = i
        for k in range(int(rows[b])):
            pos = base[b] + k
            out["row_request"][i], out["position"][i] = b, pos
            out["slot"][i] = int(table[b, pos // page]) * page + pos % page
            i += 1
    out["row_offset"][B] = i
    return dict(out, length=np.array(base, np.int32), held=np.array(need, np.int32),
                free_state=np.array([first % cap, count - sum(take) + sum(give)], np.int32))


def e4m3_values():
    """The finite non-negative values of the 8-bit type, ascending."""
    sub = np.arange(8) * 2.0 ** -9
    normal = [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return np.concatenate([sub, normal[:-1]])             # the last code is not a number


def to_e4m3(x):
    """Nearest value (ties to the even code), beyond the largest the largest, NaN kept."""
    x = np.asarray(x, np.float64)
    grid = e4m3_values()
    a = np.minimum(np.abs(x), grid[-1])
    hi = np.searchsorted(grid, np.where(np.isnan(a), 0.0, a)).clip(1, len(grid) - 1)
    lo = hi - 1
    dlo, dhi = a - grid[lo], grid[hi] - a
    pick = np.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isnan(x), x, np.copysign(grid[pick], x))


def write_kv(k, v, slot, k_cache, v_cache, k_scale=None, v_scale=None):
    """Copies of the caches [num_blocks, Hkv, page, D] (values) with the rows stored.  The
    quotient by a scale is formed in float32, as the call defines it."""
    kc, vc = k_cache.copy(), v_cache.copy()
    page = kc.shape[2]
    for i, s in enumerate(slot):
        if s < 0:
            continue
        for x, cache, scale in ((k, kc, k_scale), (v, vc, v_scale)):
            row = x[i]
            if scale is not None:
                with np.errstate(all="ignore"):
                    row = to_e4m3(row.astype(np.float32) / scale.astype(np.float32)[:, None])
            cache[s // page, :, s % page] = row
    return kc, vc


def paged_attention(q, row_offset, length, block_table, k_cache, v_cache, scale, window=0, k_scale=None,
                    v_scale=None):
    """out [n, Hq, D] and lse [n, Hq]; weight [n, Hq, D] = sum_j p_j |v_j|, size [n, Hq] = the
    largest sum_d |scale q_d k_jd| and keys [n] = visible keys, for the error bound."""
    n, Hq, D = q.shape
    Hkv, page = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    out, weight = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, size, keys = np.full((n, Hq), -np.inf), np.zeros((n, Hq)), np.zeros(n, np.int64)
    for b in range(len(length)):
        for i in range(int(row_offset[b]), int(row_offset[b + 1])):
            pos = int(length[b]) + i - int(row_offset[b])
            lo = max(0, pos - window + 1) if window else 0
            at = np.arange(lo, pos + 1)
            ids = block_table[b, at // page]
            keys[i] = len(at)
            K, V = k_cache[ids, :, at % page], v_cache[ids, :, at % page]          # [keys, Hkv, D]
            for h in range(Hq):
                k, v = K[:, h // G], V[:, h // G]
                if k_scale is not None:
                    k, v = k * float(k_scale[h // G]), v * float(v_scale[h // G])
                s = scale * (k @ q[i, h])
                m = s.max()
                m = 0.0 if m == -np.inf else m
                e = np.exp(s - m)
                z = e.sum()
                if z == 0:
                    continue
                lse[i, h] = m + np.log(z)
                out[i, h] = (e / z) @ v
                weight[i, h] = (e / z) @ np.abs(v)
                size[i, h] = abs(scale) * (np.abs(k) @ np.abs(q[i, h])).max()
    return dict(out=out, lse=lse, weight=weight, size=size, keys=keys)


def adjust_logits(logits, out, history=None, prompt_len=None, history_len=None, draft=None, ell=None,
                  repetition=None, frequency=None, presence=None, bias_token=None, bias_value=None, mask_row=None,
                  mask=None):
    """`out` with the wanted rows replaced by the adjusted ones (float64)."""
    B, R, V = logits.shape
    y = out.astype(np.float64).copy()
    for b in range(B):
        p = int(prompt_len[b]) if prompt_len is not None else 0
        h = int(history_len[b]) if history_len is not None else 0
        prompt, output = (list(history[b, :p]), list(history[b, p:h])) if history is not None else ([], [])
        for k in range(R if ell is None else int(ell[b]) + 1):
            said = output + (list(draft[b, :k]) if draft is not None else [])
            x = logits[b, k].astype(np.float64).copy()
            for v in set(prompt) | set(said):
                if repetition is not None:
                    x[v] = x[v] / float(repetition[b]) if x[v] > 0 else x[v] * float(repetition[b])
            for v in set(said):
                if frequency is not None:
                    x[v] -= float(frequency[b]) * said.count(v)
                if presence is not None:
                    x[v] -= float(presence[b])
            if bias_token is not None:
                for t, a in zip(bias_token[b], bias_value[b]):
                    if t >= 0:
                        x[t] += float(a)
            if mask_row is not None and mask_row[b, k] >= 0:
                words = mask[mask_row[b, k]].astype(np.int64) & 0xFFFFFFFF
                v = np.arange(V)
                x[((words[v // 32] >> (v % 32)) & 1) == 0] = -np.inf
            y[b, k] = x
    return y
