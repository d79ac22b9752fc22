// append_q8.cu -- the launches of the append to an 8-bit cache (append_q8_kernel.cuh) and
// its e4m3 instances; the int8 ones are in append_q8_int8.cu.
#include <algorithm>

#include "append_q8_kernel.cuh"

namespace dattn {

const void *append_q8_int8_fn(int width, bool fixed, int hp);
const void *append_token_int8_fn(int width);

namespace {

// Channels of an item, one by one where smaller items would need more than a warp's
// lanes for a row.
int append_width(int rope_dims, int D) {
    const int width = item_width(rope_dims, D);
    return D > 32 * width ? 1 : width;
}

cudaError_t launch_append_token(const Q8AppendArgs &a, int kv, cudaStream_t stream) {
    const int width = append_width(a.rope.rope_dims, a.D);
    TokenGrid gr{};
    gr.items_k = row_items(a.rope.rope_dims, a.D, width);
    gr.items_v = row_items(0, a.D, width);
    gr.lanes = 1;
    while (gr.lanes < std::max(gr.items_k, gr.items_v)) gr.lanes *= 2;
    const long long chunks = ((a.H + 2LL * a.kv_heads) * gr.lanes + kThreads - 1) / kThreads;
    const long long blocks = a.B * chunks;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    gr.chunks = static_cast<int>(chunks);
    const void *fn = kv == kKvE4m3 ? token_kernel_of<kKvE4m3>(width) : append_token_int8_fn(width);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {const_cast<Q8AppendArgs *>(&a), &gr};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_append_q8(const Q8AppendArgs &a, int kv, int sms, cudaStream_t stream) {
    if (a.offsets == nullptr) return launch_append_token(a, kv, stream);
    const int rd = a.rope.rope_dims;
    RopeGrid qgr{};
    int hp = 1;
    bool fixed = false;
    const int width = append_width(rd, a.D);
    // of q two heads per thread, of its smaller items four (8192 tokens of 32 query and 8
    // key/value heads of 96 channels, 24 of them rotated: 44 us with 4, 48 with 2, 62 with 1)
    if (!rope_grid(a.tokens, a.H, a.D, rd, width == 16 ? 2 : 4, sms, &qgr, &hp, width, &fixed))
        return cudaErrorInvalidValue;
    AppendGrid gr{};
    gr.items_k = row_items(rd, a.D, width);
    gr.items_v = row_items(0, a.D, width);
    gr.lanes = 1;
    while (gr.lanes < std::max(gr.items_k, gr.items_v)) gr.lanes *= 2;
    // rows of a block: side by side in the lanes of a warp first, then in more warps.  (For
    // the mean of the new tokens of a sequence, where that is less: 64 sequences that
    // bring 127 tokens, most of them one, 33 us against 6.8.)
    gr.rows = 1;
    while (gr.rows < a.scale_block && 2 * gr.rows * gr.lanes <= 32) gr.rows *= 2;
    gr.warps = 1;
    while (gr.warps < kWarps && gr.warps * gr.rows < a.scale_block) gr.warps *= 2;
    gr.groups_per_warp = 32 / (gr.lanes * gr.rows);
    // warps enough for all heads, at most the CTA's
    gr.set = gr.warps;
    while (gr.set < kWarps && kHeads * gr.groups_per_warp * (gr.set / gr.warps) < a.kv_heads) gr.set *= 2;
    gr.heads_per_set = kHeads * gr.groups_per_warp * (gr.set / gr.warps);
    gr.head_chunks = (a.kv_heads + gr.heads_per_set - 1) / gr.heads_per_set;
    // Two blocks per window at most, one token per window when sequences are short; smaller
    // where two blocks would leave warps idle, since a set takes its blocks one after another
    // (301 tokens of 13 sequences, 8 heads: 12.5 us with windows of 16 tokens, 8.8 with 1).
    // Two blocks, as taken, and one, with twice as many windows: 7050 tokens of 8 heads in
    // blocks of eight 15.4 and 21.5 us; 8192 of 32 on 8 heads 36.4 and 36.7.
    const int sets = kWarps / gr.set;
    const long long mean = std::max(1LL, a.tokens / a.B);
    gr.window = static_cast<int>(std::min<long long>(mean, 2LL * a.scale_block));
    while (gr.window > 1 && a.tokens / gr.window * gr.head_chunks < static_cast<long long>(sms) * sets)
        gr.window = (gr.window + 1) / 2;
    const long long jobs = (a.tokens + gr.window - 1) / gr.window * gr.head_chunks;
    const long long kv_ctas = (jobs + sets - 1) / sets * 2;
    if (jobs > 0x7fffffffLL) return cudaErrorInvalidValue;
    gr.jobs = static_cast<unsigned>(jobs);
    // q by one CTA of each SM's two slots
    const long long q_ctas = std::min<long long>(qgr.tiles, sms);
    if (kv_ctas + q_ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    gr.kv_ctas = static_cast<unsigned>(kv_ctas);
    gr.q_ctas = static_cast<unsigned>(q_ctas);
    RopeArgs q{};
    q.x = a.q;
    q.out = a.q_out;
    q.offsets = a.offsets;
    q.cur_pos = a.cur_pos;
    q.B = a.B;
    q.x_stride = a.q_stride;
    q.out_stride = static_cast<long long>(a.H) * a.D;
    q.tokens = a.tokens;
    q.H = a.H;
    q.D = a.D;
    Instance in = instance_of<kKvE4m3>(width, fixed, hp);
    if (kv == kKvInt8) in.fn = append_q8_int8_fn(width, fixed, hp);
    const size_t smem = rope_smem(qgr, rd, width, in.ring_bytes);
    if (smem > 32 * 1024) {  // with the static part past the default limit
        const cudaError_t e =
            cudaFuncSetAttribute(in.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicSmem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(kv_ctas + q_ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {const_cast<Q8AppendArgs *>(&a), &q, &gr, &qgr};
    return cudaLaunchKernelExC(&cfg, in.fn, args);
}

}  // namespace dattn
