// Host side of the decode forward over caches of different lengths
// (decode_line.cuh): the choice of variant, the workspace and the launches.
#include <cstring>

#include "decode_line.cuh"

namespace ffpa {
namespace {

using line::exchange_bytes;
using line::kLineSmem;
using line::kMaxGroups;
using line::kMaxStages;
using line::kUnitPlaces;

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

line::LinePlan line_plan(const Problem& pb, bool shared, int Np)
{
    line::LinePlan p{};
    line::LineGeo& g = p.g;
    g.chunks = pb.D / 64;
    g.R = pb.Hq / pb.Hkv * pb.Nq;
    g.Rp = pb.B * g.R;
    const int sms = num_sms() > 0 ? num_sms() : 152;
    // The prefix of sixteen rows is read by this kernel at HBM's rate; with more,
    // it passes once per sixteen and the tensor cores are faster (D = 512, eight
    // heads of 16384 keys: 64 rows 74 us), but for prefixes so short that their
    // launch costs more than eight tiles per SM do.
    const bool split = shared && Np > 0 && g.Rp > 16 &&
                       static_cast<long long>(pb.Hkv) * ((g.Rp + 15) / 16) * ((Np + 31) / 32) > 8LL * sms;
    const int most = shared && !split ? max(g.R, min(g.Rp, 32)) : g.R;
    const int mt = g.chunks > 8 || most <= 16 ? 1 : 2;
    g.rows = 16 * mt;
    g.rblocks = (g.R + g.rows - 1) / g.rows;
    // Eight compute warps and tiles of 32 keys where they make one or two groups
    // without rest; else fifteen and tiles of 16 (tile_keys).
    g.warps = min(g.chunks, 8);
    g.many = mt == 1 && (g.warps < 4 || 8 % g.warps != 0);
    g.groups = min(kMaxGroups, (g.many ? 15 : 8) / g.warps);
    g.shift = g.chunks <= 8 && !g.many ? 5 : 4;
    if (split) {
        p.prefix = pb;
        p.prefix.B = 1;
        p.prefix.Hq = pb.Hkv;
        p.prefix.Nq = g.Rp;
        p.prefix.Nkv = Np;
        p.prefix.causal = 0;
        g.splits = xchg_splits(p.prefix);
        const int tiles = (Np + 127) / 128;
        g.split_keys = (tiles + g.splits - 1) / g.splits * 128;
    } else if (shared) {
        g.rblocks_p = (g.Rp + g.rows - 1) / g.rows;
        g.tiles_p = (Np + (1 << g.shift) - 1) >> g.shift;
        if (g.tiles_p == 0) g.rblocks_p = 0;
    }
    g.stage_bytes = 2 * g.chunks * 128 << g.shift;
    const int exchange = g.groups * exchange_bytes(g.warps, mt, (1 << g.shift) / 8);
    const int budget = kLineSmem - exchange;
    g.stages = min(kMaxStages, budget / (g.groups * g.stage_bytes));
    p.smem = g.groups * g.stages * g.stage_bytes + exchange;
    p.ctas = sms;
    g.ranges = p.ctas * g.groups;
    g.pitch = (pb.Nkv + 3) & ~3;
    const size_t rows_all = static_cast<size_t>(pb.B) * pb.Hq * pb.Nq, D = pb.D;
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t here = at;
        at = up256(at + floats * sizeof(float));
        return here;
    };
    p.o_cut = take(2 * static_cast<size_t>(g.ranges) * g.rows * D);
    p.l_cut = take(2 * static_cast<size_t>(g.ranges) * g.rows);
    p.l_whole = take(rows_all);
    p.before = take(static_cast<size_t>(pb.B) + 1);  // (as wide as a float)
    if (shared) {
        p.o_whole = take(rows_all * D);
        p.o_whole_p = take(g.rblocks_p ? rows_all * D : 0);
        p.l_whole_p = take(g.rblocks_p ? rows_all : 0);
        p.o_split = take(g.splits * rows_all * D);
        p.l_split = take(g.splits * rows_all);
        p.q_rows = take(g.splits ? rows_all * D / 2 : 0);
    } else {
        p.scores = take(rows_all * g.pitch);
    }
    p.total = at;
    return p;
}

}  // namespace

bool line_fits(const Problem& pb, bool shared, int Np)
{
    const long long R = static_cast<long long>(pb.Hq / pb.Hkv) * pb.Nq;
    if (R * pb.B > 0x7fffffffLL) return false;
    // a row is joined by up to eight warps, numbered in 32 bits; key tiles of a range are counted in 31
    const long long units = static_cast<long long>(pb.B) * pb.Hkv * ((R + 15) / 16);
    const long long tiles = units * (pb.Nkv / 16 + 1 + kUnitPlaces) +
        (shared ? static_cast<long long>(pb.Hkv) * ((R * pb.B + 15) / 16) * (Np / 16 + 1 + kUnitPlaces) : 0);
    return tiles < 0x7fffffffLL && R * pb.B * pb.Hkv < 0x10000000LL;
}

size_t line_workspace_bytes(const Problem& pb, bool shared, int Np)
{
    if (pb.B <= 0 || pb.Hq <= 0 || pb.Nq <= 0) return 0;
    return line_plan(pb, shared, Np).total;
}

cudaError_t launch_line(const LineArgs& args, void* workspace, size_t workspace_bytes, size_t* need, cudaStream_t s)
{
    LineArgs a = args;
    const Problem& pb = a.f.pb;
    line::LinePlan p = line_plan(pb, a.shared, a.Np);
    line::LineGeo& g = p.g;
    *need = p.total;
    if (workspace_bytes < p.total) return cudaErrorInvalidValue;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
    g.o_cut = at(p.o_cut);
    g.l_cut = at(p.l_cut);
    g.o_whole = at(p.o_whole);
    g.l_whole = at(p.l_whole);
    g.o_whole_p = at(p.o_whole_p);
    g.l_whole_p = at(p.l_whole_p);
    g.before = reinterpret_cast<int*>(ws + p.before);
    g.scores = at(p.scores);
    g.o_split = at(p.o_split);
    g.l_split = at(p.l_split);
    g.q_rows = reinterpret_cast<uint16_t*>(ws + p.q_rows);
    CUtensorMap m[4];
    std::memset(m, 0, sizeof(m));
    Problem pp = pb;  // the prefix as one batch entry
    pp.B = 1;
    pp.Nkv = a.Np;
    // maps of sides without keys are never read
    if (pb.Nkv > 0 && (!make_slab_map(&m[0], a.f.k, pb, true, a.f.bf16, 1 << g.shift, g.chunks, pb.vk) ||
                       !make_slab_map(&m[1], a.f.v, pb, true, a.f.bf16, 1 << g.shift, g.chunks, pb.vv)))
        return cudaErrorInvalidValue;
    if (g.rblocks_p && (!make_slab_map(&m[2], a.kp, pp, true, a.f.bf16, 1 << g.shift, g.chunks, a.vkp) ||
                        !make_slab_map(&m[3], a.vp, pp, true, a.f.bf16, 1 << g.shift, g.chunks, a.vvp)))
        return cudaErrorInvalidValue;
    cudaError_t e = a.f.bf16 ? line::run_line<true>(a, p, m, s) : line::run_line<false>(a, p, m, s);
    if (e != cudaSuccess) return e;
    if (g.splits) {
        XArgs x{};
        x.pb = p.prefix;
        const long long D = pb.D;
        x.pb.vq = View{0, g.Rp * D, D};
        x.pb.vk = a.vkp;
        x.pb.vv = a.vvp;
        x.bf16 = a.f.bf16;
        x.q = g.q_rows;
        x.k = a.kp;
        x.v = a.vp;
        x.ctl = a.f.ctl;
        x.pdl = 1;
        x.splits = g.splits;
        x.split_keys = g.split_keys;
        x.split_rows = g.R;
        x.split_nq = pb.Nq;
        x.split_causal = pb.causal;
        x.split_lens = a.lens;
        x.split_most = pb.Nkv;
        x.o_part = g.o_split;
        x.l_part = g.l_split;
        if ((e = launch_xchg(XOP_FWD, x, s)) != cudaSuccess) return e;
    }
    return a.f.bf16 ? line::run_join<true>(a, p, s) : line::run_join<false>(a, p, s);
}

}  // namespace ffpa
