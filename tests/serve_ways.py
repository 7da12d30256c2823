"""Which way s2o_attention_paged takes a call, read off its workspace size: each
way of the host's rule lays out other buffers (a device of 148 SMs, and without
one the same number is taken).  A test that means to reach a way pins it here."""
import score_keys_pooled_b200 as s2o

SMS = 148


def sizes(cfg):
    """{way: bytes} of the ways open to a call of this config."""
    up = lambda n: -(-n // 256) * 256
    G = cfg.Hq // cfg.Hkv
    seq_rows = min(cfg.max_q, max(cfg.Tq, 1)) * G
    R = 1 if seq_rows <= 16 else 2
    slots = lambda workers, rows: up(2 * workers * rows * 512) + up(2 * workers * rows * 8)
    rows = cfg.Tq * cfg.Hq
    dense = 2 * (up(rows * 512) + up(rows * 8))
    head, meta, split = up(2 * 16), up(cfg.Tq * cfg.Hkv * 16), up(SMS * 16)
    tile, decode = slots(SMS, 256), slots(SMS * 8 // R, 16 * R)
    if seq_rows > 32:
        return {"chunks walk": head + split + tile, "chunks items": head + meta + dense + tile}
    name = "decode%d " % R
    return {name + "walk": head + meta + decode, name + "items": head + meta + dense + decode,
            name + "tiles": head + meta + dense + tile + decode}


def way(cfg):
    """The way a call of this config takes; without a prefix "walk" stands for
    own keys alone."""
    n = s2o.attention_paged_workspace_size(cfg)
    found = [w for w, b in sizes(cfg).items() if b == n]
    assert len(found) == 1, (n, sizes(cfg))
    return found[0]
